// Normalisation of queries and keys per head with the position rotation in the same pass, its
// gradient, and the append of keys and values to a paged cache (include/fa.h, fa_qk_norm_rope).
//
// Forward, for each token and head (x: the head's d values, w: the norm's weight):
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,
//   and for the pairs (a, b) of the leading rot_dim values of y, at the token's position,
//   (a, b) -> (a cos - b sin, b cos + a sin).
// Gradient, with g the incoming gradient turned back (the rotation's transpose) and xh = x r:
//   dw = sum over tokens and heads of g xh,   dx = r (g w - xh mean(g w xh)).
// Statistics and products are fp32; each output is rounded once to the 16-bit type.
//
// Both are streams: 2 (forward) or 3 (gradient) passes over the rows, nothing to reuse but
// the angles and the weights, so HBM bounds them and what counts is the bytes in flight.  One
// CTA per SM of 12 warps, each on its own: a warp walks over units (some rows of one token, of q,
// or of k and v) and keeps the next units' rows and angles on their way into its own shared-memory
// buffers by bulk copies, so that the loads do not wait for its arithmetic nor take registers.
// (Loads into registers, 4 row batches a warp at 16 warps per SM, reached 58 % of the copy rate.)
// A row is held by d / 16 lanes (16 at d = 192, four of them idle): a lane has two 8-value units
// that rotate with each other (unit p and p + rot / 16 when pairs lie half the rotated part
// apart; both members of each pair in one unit when they are adjacent), so the rotation needs no
// exchange between lanes, and the row sums are a few shuffles.
//
// The EXT instantiations take several position axes and leave the norm out on demand.  A token's
// angles are then no row of the tables: pair j's come from the row of its own axis's position, so
// the warp gathers them, four bytes a lane, by asynchronous copies that arrive on the unit's barrier
// like its rows.  Without the norm y is x turned, and dx is dy turned back, which the forward kernel does as
// well: x is not read.  (16384 tokens, 32 / 8 heads of 128, three axes: with the norm 60.6 us, gradient without it
// 59.7, 50.3 at the copy rate; angles gathered without their positions asked for a unit ahead 64.2 / 64.0.)
#include "rope.cuh"

namespace fa {
namespace {

// 12 warps of two 8 KB buffers fill the shared memory.  Measured, forward / gradient of 16384
// tokens of 32 + 8 heads of 128 and append of 8192 tokens of 16 + 2 heads of 256 (with v in units of
// its own), us: 54.7 / 85.1 / 32.4; 8 warps of three 64.0 / 103.0 / 39.6; 12 of three 4 KB ones 60.5 / 99.5 / 37.0; 16 of two
// 4 KB ones 58.1 / 101.1 / 32.8.  (At the copy rate: 50.1 / 74.8 / 25.0.)
constexpr int kWarps = 12;
constexpr int kBufs = 2;           // units in flight per warp

// Shared memory of a warp's buffer: rows (kUnitBytes), cos and sin of the token
template <int D>
struct __align__(128) RowBuf {
    uint8_t rows[kUnitBytes];
    float cos[D / 2], sin[D / 2];
};
struct RowMeta {
    int pos, slot;
};
template <int D>
struct WarpSmem {
    RowBuf<D> buf[kBufs];
    uint64_t full[kBufs];
    RowMeta meta[kBufs];
};

// The position of axis x of token t as it stands (lanes x < axes; `on`; 0 in the others), and, when it is
// there, in every lane whether the token has a row of the tables on each axis: padding (-1 on some axis)
// and positions outside the tables, which set the status, have none.
__device__ __forceinline__ int axis_position(const RopeArgs& a, long t, int x, bool on) {
    return !on ? 0 : a.positions ? a.positions[x * (long)a.T + t] : (int)((unsigned)t % (unsigned)a.seq_len);
}
__device__ __forceinline__ bool on_every_axis(const RopeArgs& a, int pos, bool on) {
    const bool bad = on && (pos < 0 || pos >= a.max_pos);
    if (bad && pos != -1 && a.status) atomicCAS(a.status, 0, kStatusDeviceCheck);
    return !__any_sync(0xffffffffu, bad);
}

// The axes of the pairs lane, lane + 32, ... (a byte each).
__device__ __forceinline__ uint32_t lane_axes(const RopeArgs& a, int lane) {
    uint32_t x = 0;
    if (a.axes > 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) x |= (uint32_t)a.pair_axis[lane + 32 * i] << (8 * i);
    return x;
}

// Starts the copies of a token's angles (pos: lane x's position of axis x), each pair from the row of
// its axis; every lane arrives on the barrier when its own have landed.
__device__ __forceinline__ void gather_angles(const RopeArgs& a, uint32_t axes, int pos, float* cs, float* sn, uint64_t* bar) {
    const int lane = threadIdx.x & 31, half = a.rot / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = lane + 32 * i;
        const int at = __shfl_sync(0xffffffffu, pos, (axes >> (8 * i)) & 0xff);
        if (j < half) {
            copy4_async(cs + j, a.cos + (long)at * half + j);
            copy4_async(sn + j, a.sin + (long)at * half + j);
        }
    }
    mbar_arrive_copies(bar);
}

// The token's row of the angle tables, or -1: a padding token (position -1) or one outside the
// tables, which sets the status.
__device__ __forceinline__ int position_of(const RopeArgs& a, long t) {
    const int pos = a.positions ? a.positions[t] : (int)((unsigned)t % (unsigned)a.seq_len);
    if (pos >= 0 && pos < a.max_pos) return pos;
    if (pos != -1 && a.status) atomicCAS(a.status, 0, kStatusDeviceCheck);
    return -1;
}

// The walk of a warp over units u, u + step, ...: unit x of token t, x = u % per_token.
struct UnitWalk {
    long t, dt;
    int x, dx, per_token;
    __device__ __forceinline__ UnitWalk(unsigned first, unsigned step, unsigned per)
        : t(first / per), dt(step / per), x((int)(first % per)), dx((int)(step % per)), per_token((int)per) {}
    __device__ __forceinline__ void next() {
        t += dt;
        x += dx;
        if (x >= per_token) {
            x -= per_token;
            ++t;
        }
    }
};

// Bits of the buffers with copies on their way (lane 0's; the others leave it alone).  What a warp does when
// a wait ran out: the status, and then (with the fixed limit) the wait for the copies under way, which
// must not land in shared memory that is not the warp's any more.
template <class S>
__device__ __forceinline__ void give_up(S& s, uint32_t flight, uint32_t phase, int* status) {
    if ((threadIdx.x & 31) == 0) {
        if (status) atomicCAS(status, 0, kStatusTimeout);
        for (int b = 0; b < kBufs; ++b)
            if ((flight >> b) & 1) mbar_wait_quiet(&s.full[b], (phase >> b) & 1);
    }
    __syncwarp();
}

// One run of units: `heads` rows of each token in groups of `rows`.
__device__ __forceinline__ int groups_of(int heads, int rows) { return (heads + rows - 1) / rows; }

template <int D, bool F16, bool ADJ, bool EXT>
__global__ void __launch_bounds__(32 * kWarps, 1) norm_rope_kernel(const RopeArgs a) {
    using C = RowCfg<D>;
    constexpr int LANES = C::LANES, ROWS = C::ROWS;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % LANES, lr = lane / LANES;
    WarpSmem<D>& s = reinterpret_cast<WarpSmem<D>*>(smem_raw)[warp];
    const bool on = li < C::PAIRS;
    const int gq = groups_of(a.h_q, a.unit_rows), per_token = gq + groups_of(a.h_kv, a.kv_rows);
    const unsigned n_warps = (unsigned)a.warps, me = blockIdx.x * kWarps + warp;
    // a unit's kind (0 q, 1 k and, in an append, v), first row and rows
    auto unit = [&](int x, int& kind, int& r0, int& rows) {
        kind = x < gq ? 0 : 1;
        r0 = kind ? (x - gq) * a.kv_rows : x * a.unit_rows;
        rows = kind ? min(a.kv_rows, a.h_kv - r0) : min(a.unit_rows, a.h_q - r0);
    };
    UnitWalk ahead(me, n_warps, per_token), now = ahead;
    if (me >= n_warps) ahead.t = now.t = a.T;
    int next_pos = -1, next_slot = -1;  // of the unit `ahead` (lane 0; EXT: next_pos of axis `lane`)
    uint32_t flight = 0;                // buffers with copies on their way (lane 0)
    const uint32_t axes = EXT ? lane_axes(a, lane) : 0;
    const bool has_axis = lane < max(a.axes, 1);
    auto look = [&]() {
        if constexpr (EXT) {
            if (ahead.t < a.T) next_pos = axis_position(a, ahead.t, lane, has_axis);
            if (lane == 0 && ahead.t < a.T && a.slots && ahead.x >= gq) {
                next_slot = a.slots[ahead.t];
                if (next_slot >= a.num_slots || next_slot < -1) {
                    if (a.status) atomicCAS(a.status, 0, kStatusDeviceCheck);
                    next_slot = -1;
                }
            }
            return;
        }
        if (lane == 0 && ahead.t < a.T) {
            next_pos = position_of(a, ahead.t);
            if (a.slots && ahead.x >= gq) {
                next_slot = a.slots[ahead.t];
                if (next_slot >= a.num_slots || next_slot < -1) {
                    if (a.status) atomicCAS(a.status, 0, kStatusDeviceCheck);
                    next_slot = -1;
                }
            }
        }
    };
    // starts the copies of the unit `ahead` into buffer b and moves on
    auto issue = [&](int b) {
        if (EXT && ahead.t < a.T) {
            if (on_every_axis(a, next_pos, has_axis)) gather_angles(a, axes, next_pos, s.buf[b].cos, s.buf[b].sin, &s.full[b]);
            else next_pos = -1;
        }
        if (lane == 0 && ahead.t < a.T) {
            s.meta[b] = RowMeta{next_pos, next_slot};
            if (next_pos >= 0) {
                int kind, r0, rows;
                unit(ahead.x, kind, r0, rows);
                const bool with_v = kind && a.v;
                const uint16_t* src = (kind ? a.k + ahead.t * a.k_stride : a.q + ahead.t * a.q_stride) + (long)r0 * D;
                const uint32_t bytes = (uint32_t)rows * D * 2, angle = EXT ? 0u : (uint32_t)a.rot * 2;
                flight |= 1u << b;
                mbar_expect_tx(&s.full[b], (with_v ? 2 : 1) * bytes + 2 * angle);
                bulk_load(s.buf[b].rows, src, bytes, &s.full[b]);
                if (with_v) bulk_load(s.buf[b].rows + kUnitBytes / 2, a.v + ahead.t * a.v_stride + (long)r0 * D, bytes, &s.full[b]);
                if (angle) {
                    bulk_load(s.buf[b].cos, a.cos + (long)next_pos * (a.rot / 2), angle, &s.full[b]);
                    bulk_load(s.buf[b].sin, a.sin + (long)next_pos * (a.rot / 2), angle, &s.full[b]);
                }
            }
        }
        ahead.next();
        look();
    };
    if (lane == 0) {
        for (int b = 0; b < kBufs; ++b) mbar_init(&s.full[b], EXT ? 33 : 1);  // (lane 0's arrival, and the lanes' copies)
        fence_mbar_init();
    }
    __syncwarp();
    look();
    for (int b = 0; b < kBufs; ++b) issue(b);
    if (EXT && a.beside) allow_next_kernel();
    int u0, u1;
    lane_units<D, ADJ>(on ? li : 0, a.rot, u0, u1);
    float2 wq[8], wk[8];
    load_weight<F16>(a, a.wq, u0, u1, wq);
    load_weight<F16>(a, a.wk, u0, u1, wk);
    __syncwarp();
    uint32_t phase = 0;  // bit b: the parity buffer b's next copies complete
    for (int b = 0; now.t < a.T; now.next(), b = b + 1 == kBufs ? 0 : b + 1) {
        const RowMeta meta = s.meta[b];
        int kind, r0, rows;
        unit(now.x, kind, r0, rows);
        uint16_t* out0;
        if constexpr (EXT)
            out0 = kind == 0 ? a.q_out + now.t * a.dq_stride + (long)r0 * D : a.k_out ? a.k_out + now.t * a.dk_stride + (long)r0 * D : nullptr;
        else out0 = kind == 0 ? a.q_out + (now.t * a.h_q + r0) * D : a.k_out ? a.k_out + (now.t * a.h_kv + r0) * D : nullptr;
        if (meta.pos >= 0) {
            if (!__all_sync(0xffffffffu, mbar_wait_within(&s.full[b], (phase >> b) & 1, a.wait_ns))) {
                give_up(s, flight, phase, a.status);
                return;
            }
            phase ^= 1u << b;
            flight &= ~(1u << b);
            const uint8_t* in = s.buf[b].rows;
            const bool cached = kind && meta.slot >= 0;
            const long in_cache = ((long)meta.slot * a.h_kv + r0) * D;
            uint16_t* out1 = cached ? a.k_cache + in_cache : nullptr;
            if (cached)
                for (int y = lane; y < rows * D / 8; y += 32)
                    reinterpret_cast<uint4*>(a.v_cache + in_cache)[y] = reinterpret_cast<const uint4*>(in + kUnitBytes / 2)[y];
            if (out0 || out1) {
                Angles<ADJ> ang;
                ang.load(s.buf[b].cos, s.buf[b].sin, u0, u1, a.rot);
                if (EXT && a.back) ang.turn_round();
                // (two row batches at a time, so that one's sums and roots hide behind the other's)
#pragma unroll 2
                for (int r = lr; r < rows + lr; r += ROWS) {
                    const bool live = on && r < rows;
                    float2 v[8];
                    {
                        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
                        if (live) {
                            x0 = *reinterpret_cast<const uint4*>(in + r * (D * 2) + 16 * u0);
                            x1 = *reinterpret_cast<const uint4*>(in + r * (D * 2) + 16 * u1);
                        }
                        widen8<F16>(x0, v);
                        widen8<F16>(x1, v + 4);
                    }
                    float2 ss = __fmul2_rn(v[0], v[0]);
#pragma unroll
                    for (int e = 1; e < 8; ++e) ss = __ffma2_rn(v[e], v[e], ss);
                    float rs = rsqrtf(row_sum<LANES>(ss.x + ss.y) * (1.f / D) + a.eps);
                    if (EXT && a.no_norm) rs = 1.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = __fmul2_rn(v[e], kind ? wk[e] : wq[e]);
                    ang.template turn<false, EXT>(v, (ADJ ? 8 : 16) * u0 < a.rot, 8 * u1 < a.rot);
                    const float2 rs2 = make_float2(rs, rs);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = __fmul2_rn(v[e], rs2);
                    const uint4 y0 = narrow8<F16>(v), y1 = narrow8<F16>(v + 4);
                    if (live && out0) {
                        *reinterpret_cast<uint4*>(out0 + r * D + 8 * u0) = y0;
                        *reinterpret_cast<uint4*>(out0 + r * D + 8 * u1) = y1;
                    }
                    if (live && out1) {
                        *reinterpret_cast<uint4*>(out1 + r * D + 8 * u0) = y0;
                        *reinterpret_cast<uint4*>(out1 + r * D + 8 * u1) = y1;
                    }
                }
            }
        } else if (a.zero_skipped && out0) {
            for (int y = lane; y < rows * D / 8; y += 32) reinterpret_cast<uint4*>(out0)[y] = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();  // the buffer has been read
        issue(b);
        __syncwarp();
    }
}

// Gradient: the same walk, over the query rows and then over the key rows, with dy beside x in
// the buffer and the weight gradient of the lane's own values in registers.  Each CTA adds its
// warps' sums in a fixed order and stores them as one row of the workspace; norm_rope_dw_kernel
// adds the rows, again in a fixed order, so the gradients are the same bits from call to call.
// The sums are fp32: a term carries fp32 roundings already, and with a lane's chain followed by trees over
// lanes, warps and CTAs the error stays within 2^-16 of the sum of the terms' sizes.
template <int D, bool F16, bool ADJ, bool EXT>
__global__ void __launch_bounds__(32 * kWarps, 1) norm_rope_bwd_kernel(const RopeArgs a) {
    using C = RowCfg<D>;
    constexpr int LANES = C::LANES, ROWS = C::ROWS;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % LANES, lr = lane / LANES;
    WarpSmem<D>& s = reinterpret_cast<WarpSmem<D>*>(smem_raw)[warp];
    const bool on = li < C::PAIRS;
    int u0, u1;
    lane_units<D, ADJ>(on ? li : 0, a.rot, u0, u1);
    if (lane == 0) {
        for (int b = 0; b < kBufs; ++b) mbar_init(&s.full[b], EXT ? 33 : 1);  // (lane 0's arrival, and the lanes' copies)
        fence_mbar_init();
    }
    __syncwarp();
    const unsigned n_warps = (unsigned)a.warps, me = blockIdx.x * kWarps + warp;
    uint32_t phase = 0, flight = 0;
    bool failed = false;
    const uint32_t axes = EXT ? lane_axes(a, lane) : 0;
    const bool has_axis = lane < max(a.axes, 1);
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const int heads = kind ? a.h_kv : a.h_q;
        const uint16_t* xs = kind ? a.k : a.q;
        const uint16_t* gs = kind ? a.dk_out : a.dq_out;
        uint16_t* ds = kind ? a.dk : a.dq;
        const long xstride = kind ? a.k_stride : a.q_stride, dstride = kind ? a.dk_stride : a.dq_stride;
        float2 w[8], dw[8];
        load_weight<F16>(a, kind ? a.wk : a.wq, u0, u1, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = make_float2(0.f, 0.f);
        UnitWalk ahead(me, n_warps, groups_of(heads, a.unit_rows)), now = ahead;
        if (me >= n_warps) ahead.t = now.t = a.T;
        int next_pos = -1;
        auto look = [&]() {
            if constexpr (EXT) {
                if (ahead.t < a.T) next_pos = axis_position(a, ahead.t, lane, has_axis);
            } else {
                if (lane == 0 && ahead.t < a.T) next_pos = position_of(a, ahead.t);
            }
        };
        auto issue = [&](int b) {
            if (EXT && ahead.t < a.T) {
                if (on_every_axis(a, next_pos, has_axis)) gather_angles(a, axes, next_pos, s.buf[b].cos, s.buf[b].sin, &s.full[b]);
                else next_pos = -1;
            }
            if (lane == 0 && ahead.t < a.T) {
                s.meta[b] = RowMeta{next_pos, 0};
                if (next_pos >= 0) {
                    const int r0 = ahead.x * a.unit_rows, rows = min(a.unit_rows, heads - r0);
                    const uint32_t bytes = (uint32_t)rows * D * 2, angle = EXT ? 0u : (uint32_t)a.rot * 2;
                    flight |= 1u << b;
                    mbar_expect_tx(&s.full[b], 2 * bytes + 2 * angle);
                    bulk_load(s.buf[b].rows, xs + ahead.t * xstride + (long)r0 * D, bytes, &s.full[b]);
                    bulk_load(s.buf[b].rows + kUnitBytes / 2, gs + (ahead.t * heads + r0) * D, bytes, &s.full[b]);
                    if (angle) {
                        bulk_load(s.buf[b].cos, a.cos + (long)next_pos * (a.rot / 2), angle, &s.full[b]);
                        bulk_load(s.buf[b].sin, a.sin + (long)next_pos * (a.rot / 2), angle, &s.full[b]);
                    }
                }
            }
            ahead.next();
            look();
        };
        if (!failed) {
            look();
            for (int b = 0; b < kBufs; ++b) issue(b);
        }
        __syncwarp();
        for (int b = 0; !failed && now.t < a.T; now.next(), b = b + 1 == kBufs ? 0 : b + 1) {
            const int r0 = now.x * a.unit_rows, rows = min(a.unit_rows, heads - r0);
            uint16_t* pd = ds + now.t * dstride + (long)r0 * D;
            if (s.meta[b].pos >= 0) {
                if (!__all_sync(0xffffffffu, mbar_wait_within(&s.full[b], (phase >> b) & 1, a.wait_ns))) {
                    give_up(s, flight, phase, a.status);
                    failed = true;  // (the CTA's sums below still need every warp)
                    break;
                }
                phase ^= 1u << b;
                flight &= ~(1u << b);
                const uint8_t *px = s.buf[b].rows, *pg = px + kUnitBytes / 2;
                Angles<ADJ> ang;
                ang.load(s.buf[b].cos, s.buf[b].sin, u0, u1, a.rot);
#pragma unroll 2
                for (int r = lr; r < rows + lr; r += ROWS) {
                    const bool live = on && r < rows;
                    float2 v[8], y[8];
                    {
                        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0, y0 = x0, y1 = x0;
                        if (live) {
                            x0 = *reinterpret_cast<const uint4*>(px + r * (D * 2) + 16 * u0);
                            x1 = *reinterpret_cast<const uint4*>(px + r * (D * 2) + 16 * u1);
                            y0 = *reinterpret_cast<const uint4*>(pg + r * (D * 2) + 16 * u0);
                            y1 = *reinterpret_cast<const uint4*>(pg + r * (D * 2) + 16 * u1);
                        }
                        widen8<F16>(x0, v);
                        widen8<F16>(x1, v + 4);
                        widen8<F16>(y0, y);
                        widen8<F16>(y1, y + 4);
                    }
                    ang.template turn<true, EXT>(y, (ADJ ? 8 : 16) * u0 < a.rot, 8 * u1 < a.rot);
                    float2 ss = __fmul2_rn(v[0], v[0]);
#pragma unroll
                    for (int e = 1; e < 8; ++e) ss = __ffma2_rn(v[e], v[e], ss);
                    // t = g x: what dw and mean(g w xh) sum
                    float2 t[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] = __fmul2_rn(y[e], v[e]);
                    float2 sg = __fmul2_rn(t[0], w[0]);
#pragma unroll
                    for (int e = 1; e < 8; ++e) sg = __ffma2_rn(t[e], w[e], sg);
                    // (a lane without a row adds nothing to dw: with eps = 0 its root would be infinite, and 0 * inf NaN)
                    const float root = rsqrtf(row_sum<LANES>(ss.x + ss.y) * (1.f / D) + a.eps), rs = live ? root : 0.f;
                    // dx = r g w - x r^3 mean(g w x)
                    const float m = -row_sum<LANES>(sg.x + sg.y) * (1.f / D) * rs * rs * rs;
                    const float2 rs2 = make_float2(rs, rs), m2 = make_float2(m, m);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dw[e] = __ffma2_rn(t[e], rs2, dw[e]);
                        y[e] = __fmul2_rn(__fmul2_rn(y[e], w[e]), rs2);
                        v[e] = __ffma2_rn(v[e], m2, y[e]);
                    }
                    if (live) {
                        *reinterpret_cast<uint4*>(pd + r * D + 8 * u0) = narrow8<F16>(v);
                        *reinterpret_cast<uint4*>(pd + r * D + 8 * u1) = narrow8<F16>(v + 4);
                    }
                }
            } else if (a.zero_skipped) {
                for (int y = lane; y < rows * D / 8; y += 32) reinterpret_cast<uint4*>(pd)[y] = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();  // the buffer has been read
            issue(b);
            __syncwarp();
        }
        // the warp's lanes with the same values, then the CTA's warps, in order (in the first buffer,
        // which no copy is under way into)
        float* part = reinterpret_cast<float*>(reinterpret_cast<WarpSmem<D>*>(smem_raw)[warp].buf[0].rows);
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = h ? dw[e].y : dw[e].x;
#pragma unroll
                for (int o = 16; o >= LANES; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (lane < C::PAIRS) part[8 * (e < 4 ? u0 : u1) + 2 * (e & 3) + h] = x;
            }
        __syncthreads();
        for (int j = threadIdx.x; j < D; j += 32 * kWarps) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) x += reinterpret_cast<const float*>(reinterpret_cast<WarpSmem<D>*>(smem_raw)[k].buf[0].rows)[j];
            a.dw_part[((long)kind * gridDim.x + blockIdx.x) * D + j] = x;
        }
        fence_proxy_async_smem();  // the next run's copies overwrite the sums
        __syncthreads();
    }
}

// dw[kind][j] = sum over the CTAs' rows; 32 columns to a CTA, 32 rows at a time.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const RopeArgs a, int n_part) {
    __shared__ float s[32][33];
    const int cols = a.d / 32, kind = blockIdx.x / cols, j = (blockIdx.x % cols) * 32 + (threadIdx.x & 31);
    const int y = threadIdx.x >> 5;
    const float* src = a.dw_part + (long)kind * n_part * a.d + j;
    float x = 0.f;
    for (int r = y; r < n_part; r += 32) x += src[(long)r * a.d];
    s[y][threadIdx.x & 31] = x;
    __syncthreads();
    x = s[threadIdx.x & 31][y];  // warp y: column y's 32 sums
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) (kind ? a.dwk : a.dwq)[(blockIdx.x % cols) * 32 + y] = x;
}

// Rows of a unit: as many as a buffer holds, fewer where that would leave warps without a unit
// (a decode step's few tokens: every warp then takes one batch of rows).
int unit_rows(int d, long rows, int most, int sms) {
    const int batch = d == 192 || d == 256 ? 2 : 512 / d;
    long r = rows / ((long)sms * kWarps) / batch * batch;
    return (int)(r < batch ? batch : r > most ? most : r);
}

template <int D>
constexpr int max_rows(bool bwd) { return bwd ? RowCfg<D>::MAX_ROWS / 2 : RowCfg<D>::MAX_ROWS; }

int unit_rows_of(int d, long rows, bool bwd, int sms) {
    const int most = d == 64 ? max_rows<64>(bwd) : d == 128 ? max_rows<128>(bwd) : d == 192 ? max_rows<192>(bwd) : max_rows<256>(bwd);
    return unit_rows(d, rows, most, sms);
}

template <int D, bool F16, bool ADJ, bool EXT>
cudaError_t launch_fwd_dfae(const RopeArgs& a, int ctas, cudaStream_t st) {
    constexpr int smem = sizeof(WarpSmem<D>) * kWarps;
    cudaError_t e = cudaFuncSetAttribute(norm_rope_kernel<D, F16, ADJ, EXT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    norm_rope_kernel<D, F16, ADJ, EXT><<<ctas, 32 * kWarps, smem, st>>>(a);
    return cudaGetLastError();
}

// Whether a call takes the instantiations with several axes, without the norm, or beside another kernel.
bool extended(const RopeArgs& a) { return a.axes > 1 || a.no_norm || a.beside || a.back; }

template <int D, bool F16, bool ADJ>
cudaError_t launch_fwd_dfa(const RopeArgs& a, int ctas, cudaStream_t st) {
    return extended(a) ? launch_fwd_dfae<D, F16, ADJ, true>(a, ctas, st) : launch_fwd_dfae<D, F16, ADJ, false>(a, ctas, st);
}

template <int D>
cudaError_t launch_fwd_d(const RopeArgs& a, int ctas, cudaStream_t st) {
    if (a.f16) return a.adjacent ? launch_fwd_dfa<D, true, true>(a, ctas, st) : launch_fwd_dfa<D, true, false>(a, ctas, st);
    return a.adjacent ? launch_fwd_dfa<D, false, true>(a, ctas, st) : launch_fwd_dfa<D, false, false>(a, ctas, st);
}

template <int D, bool F16, bool ADJ, bool EXT>
cudaError_t launch_bwd_dfae(const RopeArgs& a, int ctas, cudaStream_t st) {
    constexpr int smem = sizeof(WarpSmem<D>) * kWarps;
    cudaError_t e = cudaFuncSetAttribute(norm_rope_bwd_kernel<D, F16, ADJ, EXT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    norm_rope_bwd_kernel<D, F16, ADJ, EXT><<<ctas, 32 * kWarps, smem, st>>>(a);
    return cudaGetLastError();
}

template <int D, bool F16, bool ADJ>
cudaError_t launch_bwd_dfa(const RopeArgs& a, int ctas, cudaStream_t st) {
    const cudaError_t e = extended(a) ? launch_bwd_dfae<D, F16, ADJ, true>(a, ctas, st) : launch_bwd_dfae<D, F16, ADJ, false>(a, ctas, st);
    if (e != cudaSuccess) return e;
    norm_rope_dw_kernel<<<2 * (D / 32), 1024, 0, st>>>(a, ctas);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_bwd_d(const RopeArgs& a, int ctas, cudaStream_t st) {
    if (a.f16) return a.adjacent ? launch_bwd_dfa<D, true, true>(a, ctas, st) : launch_bwd_dfa<D, true, false>(a, ctas, st);
    return a.adjacent ? launch_bwd_dfa<D, false, true>(a, ctas, st) : launch_bwd_dfa<D, false, false>(a, ctas, st);
}

// Warps that walk: all of the grid's, less a few so that their number has no factor in common with
// the units of a token and every warp meets units of each size.
int walking_warps(int ctas, int per_token) {
    int n = ctas * kWarps;
    auto common = [](int x, int y) {
        while (y) {
            const int z = x % y;
            x = y;
            y = z;
        }
        return x;
    };
    while (n > 1 && common(n, per_token) > 1) --n;
    return n;
}

int ctas_for(long units, int sms) {
    const long need = (units + kWarps - 1) / kWarps;
    return (int)(need < 1 ? 1 : need < sms ? need : sms);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& args, int sms, cudaStream_t st) {
    RopeArgs a = args;
    a.unit_rows = unit_rows_of(a.d, (long)a.T * (a.h_q + (a.v ? 2 : 1) * a.h_kv), false, sms);
    // (keys and their values in one unit of an append, so that more bytes are in flight: 8192 tokens of
    // 16 + 2 heads of 256 30.9 us, 32.7 with units of their own)
    a.kv_rows = a.v ? unit_rows_of(a.d, (long)a.T * (a.h_q + 2 * a.h_kv), true, sms) : a.unit_rows;
    const int per_token = cdiv(a.h_q, a.unit_rows) + cdiv(a.h_kv, a.kv_rows);
    const int ctas = ctas_for((long)a.T * per_token, sms);
    a.warps = (long)a.T * per_token > (long)ctas * kWarps ? walking_warps(ctas, per_token) : ctas * kWarps;
    switch (a.d) {
        case 64: return launch_fwd_d<64>(a, ctas, st);
        case 128: return launch_fwd_d<128>(a, ctas, st);
        case 192: return launch_fwd_d<192>(a, ctas, st);
        case 256: return launch_fwd_d<256>(a, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

int norm_rope_bwd_ctas(const RopeArgs& a, int sms) {
    const int rows = unit_rows_of(a.d, (long)a.T * a.h_q, true, sms);
    return ctas_for((long)a.T * cdiv(a.h_q, rows), sms);
}

cudaError_t launch_norm_rope_bwd(const RopeArgs& args, int sms, cudaStream_t st) {
    RopeArgs a = args;
    a.unit_rows = unit_rows_of(a.d, (long)a.T * a.h_q, true, sms);
    const int ctas = norm_rope_bwd_ctas(a, sms);
    a.warps = ctas * kWarps;
    switch (a.d) {
        case 64: return launch_bwd_d<64>(a, ctas, st);
        case 128: return launch_bwd_d<128>(a, ctas, st);
        case 192: return launch_bwd_d<192>(a, ctas, st);
        case 256: return launch_bwd_d<256>(a, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
