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
// the angles and the weights, so HBM bounds them and the layout only has to keep enough
// 16-byte loads in flight.  A row is held by d / 16 lanes (4 at d = 192): a lane takes pairs of
// 8-value units that rotate with each other (unit p with p + rot / 16 when pairs lie half the
// rotated part apart, both members of each pair in one unit when they are adjacent), so the
// rotation needs no exchange between lanes, and the row sums are a few shuffles.
#include "kernels.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

template <int D>
struct RowCfg {
    static constexpr int PAIRS = D / 16;                   // pairs of 8-value units of a row
    static constexpr int LANES = D == 192 ? 4 : PAIRS;     // lanes that hold a row
    static constexpr int PPL = PAIRS / LANES;              // pairs a lane holds
    static constexpr int ROWS = 32 / LANES;                // rows of a warp at a time
    static constexpr int STEPS = D == 192 ? 2 : 4;         // row batches in flight
};

// The two units (8 values each, their index in the row) of pair i.
template <int D, bool ADJ>
__device__ __forceinline__ void pair_units(int i, int rot, int& u0, int& u1) {
    if constexpr (ADJ) {
        u0 = i;
        u1 = i + D / 16;
    } else {
        const int h = rot >> 4;  // units of half the rotated part
        if (i < h) {
            u0 = i;
            u1 = i + h;
        } else {  // behind the rotated part
            u0 = 2 * i;
            u1 = 2 * i + 1;
        }
    }
}

// cos and sin that the pair's 8 products need: value e of unit 0 (and e of unit 1) for pairs half
// the rotated part apart; members 2e, 2e + 1 of unit 0 (e < 4) and unit 1 (e >= 4) for adjacent ones.
template <bool ADJ>
__device__ __forceinline__ void load_angles(const float* row_c, const float* row_s, int u0, int u1, int rot, float* c,
                                            float* n) {
    auto four = [&](const float* src, float* dst) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(src));
        dst[0] = x.x; dst[1] = x.y; dst[2] = x.z; dst[3] = x.w;
    };
    const bool on0 = ADJ ? 8 * u0 < rot : 16 * u0 < rot, on1 = ADJ ? 8 * u1 < rot : on0;
    const int at0 = ADJ ? 4 * u0 : 8 * u0, at1 = ADJ ? 4 * u1 : 8 * u0 + 4;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        c[e] = 1.f;
        n[e] = 0.f;
    }
    if (on0) {
        four(row_c + at0, c);
        four(row_s + at0, n);
    }
    if (on1) {
        four(row_c + at1, c + 4);
        four(row_s + at1, n + 4);
    }
}

// Rotates the pair's 16 values (unit 0 in v[0..7], unit 1 in v[8..15]); BACK: by minus the angle.
template <bool ADJ, bool BACK>
__device__ __forceinline__ void turn(float* v, const float* c, const float* n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int ia = ADJ ? (e < 4 ? 2 * e : 8 + 2 * (e - 4)) : e, ib = ADJ ? ia + 1 : e + 8;
        const float a = v[ia], b = v[ib], s = BACK ? -n[e] : n[e];
        v[ia] = a * c[e] - b * s;
        v[ib] = b * c[e] + a * s;
    }
}

template <bool F16>
__device__ __forceinline__ void widen8(const uint4& x, float* v) {
    v[0] = lo16<F16>(x.x); v[1] = hi16<F16>(x.x); v[2] = lo16<F16>(x.y); v[3] = hi16<F16>(x.y);
    v[4] = lo16<F16>(x.z); v[5] = hi16<F16>(x.z); v[6] = lo16<F16>(x.w); v[7] = hi16<F16>(x.w);
}
template <bool F16>
__device__ __forceinline__ uint4 narrow8(const float* v) {
    return make_uint4(pack16<F16>(v[0], v[1]), pack16<F16>(v[2], v[3]), pack16<F16>(v[4], v[5]), pack16<F16>(v[6], v[7]));
}

// 8 weights from unit u (null: ones).
template <bool F16>
__device__ __forceinline__ void load_weight8(const RopeArgs& a, const void* w, int u, float* v) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 1.f;
    } else if (a.weight_f32) {
        const float4* src = reinterpret_cast<const float4*>(w) + 2 * u;
        const float4 x = __ldg(src), y = __ldg(src + 1);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else {
        widen8<F16>(__ldg(reinterpret_cast<const uint4*>(w) + u), v);
    }
}

// Sum over the lanes that hold a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The token's row of the angle tables, or -1: a padding token (position -1) or one outside the
// tables, which sets the status.
__device__ __forceinline__ int position_of(const RopeArgs& a, long t) {
    const int pos = a.positions ? a.positions[t] : (int)(t % a.seq_len);
    if (pos >= 0 && pos < a.max_pos) return pos;
    if (pos != -1 && a.status) atomicCAS(a.status, 0, kStatusDeviceCheck);
    return -1;
}

// One warp takes STEPS row batches of one token: the token's query rows, key rows and (append)
// value rows are numbered one after the other, ROWS of them to a batch.
template <int D, bool F16, bool ADJ>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const RopeArgs a) {
    using C = RowCfg<D>;
    constexpr int LANES = C::LANES, PPL = C::PPL, ROWS = C::ROWS, STEPS = C::STEPS;
    const int lane = threadIdx.x & 31, li = lane % LANES;
    const long task = (long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const long t = task / a.segments;
    if (t >= a.T) return;
    const int row0 = (int)(task - t * a.segments) * (ROWS * STEPS) + lane / LANES;
    const int n_rows = a.h_q + a.h_kv + (a.v ? a.h_kv : 0);
    int u0[PPL], u1[PPL];
#pragma unroll
    for (int i = 0; i < PPL; ++i) pair_units<D, ADJ>(li + LANES * i, a.rot, u0[i], u1[i]);

    // every row of the batches, all loads in flight at once
    uint4 x[STEPS][PPL][2];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int r = row0 + s * ROWS;
        const uint16_t* src = nullptr;
        if (r < a.h_q) src = a.q + t * a.q_stride + (long)r * D;
        else if (r < a.h_q + a.h_kv) src = a.k + t * a.k_stride + (long)(r - a.h_q) * D;
        else if (r < n_rows) src = a.v + t * a.v_stride + (long)(r - a.h_q - a.h_kv) * D;
#pragma unroll
        for (int i = 0; i < PPL; ++i) {
            x[s][i][0] = src ? *reinterpret_cast<const uint4*>(src + 8 * u0[i]) : make_uint4(0, 0, 0, 0);
            x[s][i][1] = src ? *reinterpret_cast<const uint4*>(src + 8 * u1[i]) : make_uint4(0, 0, 0, 0);
        }
    }
    const int pos = position_of(a, t);
    if (pos < 0) return;  // the whole warp: one token
    long slot = -1;
    if (a.slots) {
        slot = a.slots[t];
        if (slot >= a.num_slots || slot < -1) {
            if (a.status) atomicCAS(a.status, 0, kStatusDeviceCheck);
            slot = -1;
        }
    }
    float c[PPL][8], n[PPL][8];
#pragma unroll
    for (int i = 0; i < PPL; ++i)
        load_angles<ADJ>(a.cos + (long)pos * (a.rot / 2), a.sin + (long)pos * (a.rot / 2), u0[i], u1[i], a.rot, c[i], n[i]);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int r = row0 + s * ROWS;
        const bool is_q = r < a.h_q, is_v = r >= a.h_q + a.h_kv;
        float v[PPL][16], ss = 0.f;
#pragma unroll
        for (int i = 0; i < PPL; ++i) {
            widen8<F16>(x[s][i][0], v[i]);
            widen8<F16>(x[s][i][1], v[i] + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(v[i][e], v[i][e], ss);
        }
        const float rs = rsqrtf(row_sum<LANES>(ss) * (1.f / D) + a.eps);
        if (r >= n_rows) continue;
        if (!is_v) {
#pragma unroll
            for (int i = 0; i < PPL; ++i) {
                float w[16];
                load_weight8<F16>(a, is_q ? a.wq : a.wk, u0[i], w);
                load_weight8<F16>(a, is_q ? a.wq : a.wk, u1[i], w + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[i][e] *= rs * w[e];
                turn<ADJ, false>(v[i], c[i], n[i]);
                x[s][i][0] = narrow8<F16>(v[i]);
                x[s][i][1] = narrow8<F16>(v[i] + 8);
            }
        }
        uint16_t* dst[2] = {nullptr, nullptr};
        if (is_q) {
            dst[0] = a.q_out + (t * a.h_q + r) * (long)D;
        } else {
            const int h = r - a.h_q - (is_v ? a.h_kv : 0);
            if (!is_v && a.k_out) dst[0] = a.k_out + (t * a.h_kv + h) * (long)D;
            if (slot >= 0) dst[1] = (is_v ? a.v_cache : a.k_cache) + (slot * a.h_kv + h) * (long)D;
        }
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            if (!dst[o]) continue;
#pragma unroll
            for (int i = 0; i < PPL; ++i) {
                *reinterpret_cast<uint4*>(dst[o] + 8 * u0[i]) = x[s][i][0];
                *reinterpret_cast<uint4*>(dst[o] + 8 * u1[i]) = x[s][i][1];
            }
        }
    }
}

// Gradient.  The query rows and the key rows are two runs of row batches; the grid's warps
// stride over the first, then the second, keeping the weight gradient of the lane's own values
// in registers.  Each CTA adds its warps' sums in a fixed order and stores them as one row of the
// workspace; norm_rope_dw_kernel adds the rows, again in a fixed order, so the gradients are the
// same bits from call to call.
constexpr int kBwdWarps = 8;

template <int D, bool F16, bool ADJ>
__global__ void __launch_bounds__(32 * kBwdWarps) norm_rope_bwd_kernel(const RopeArgs a) {
    using C = RowCfg<D>;
    constexpr int LANES = C::LANES, PPL = C::PPL, ROWS = C::ROWS;
    __shared__ float part[kBwdWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % LANES;
    int u0[PPL], u1[PPL];
#pragma unroll
    for (int i = 0; i < PPL; ++i) pair_units<D, ADJ>(li + LANES * i, a.rot, u0[i], u1[i]);
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const int heads = kind ? a.h_kv : a.h_q;
        const uint16_t* xs = kind ? a.k : a.q;
        const uint16_t* gs = kind ? a.dk_out : a.dq_out;
        uint16_t* ds = kind ? a.dk : a.dq;
        const long xstride = kind ? a.k_stride : a.q_stride, dstride = kind ? a.dk_stride : a.dq_stride;
        float w[PPL][16], dw[PPL][16];
#pragma unroll
        for (int i = 0; i < PPL; ++i) {
            load_weight8<F16>(a, kind ? a.wk : a.wq, u0[i], w[i]);
            load_weight8<F16>(a, kind ? a.wk : a.wq, u1[i], w[i] + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) dw[i][e] = 0.f;
        }
        const long rows = (long)a.T * heads, step = (long)gridDim.x * kBwdWarps * ROWS;
        for (long base = ((long)blockIdx.x * kBwdWarps + warp) * ROWS; base < rows; base += step) {
            const long row = base + lane / LANES;
            const bool in = row < rows;
            const long t = in ? row / heads : 0;
            const long h = in ? row - t * heads : 0;
            const int pos = in ? position_of(a, t) : -1;
            const bool live = pos >= 0;
            uint4 x[PPL][2], g[PPL][2];
            float c[PPL][8], n[PPL][8];
#pragma unroll
            for (int i = 0; i < PPL; ++i) {
                const uint16_t* px = xs + t * xstride + h * D;
                const uint16_t* pg = gs + (t * heads + h) * D;
                const uint4 zero = make_uint4(0, 0, 0, 0);
                x[i][0] = live ? *reinterpret_cast<const uint4*>(px + 8 * u0[i]) : zero;
                x[i][1] = live ? *reinterpret_cast<const uint4*>(px + 8 * u1[i]) : zero;
                g[i][0] = live ? *reinterpret_cast<const uint4*>(pg + 8 * u0[i]) : zero;
                g[i][1] = live ? *reinterpret_cast<const uint4*>(pg + 8 * u1[i]) : zero;
                load_angles<ADJ>(a.cos + (long)max(pos, 0) * (a.rot / 2), a.sin + (long)max(pos, 0) * (a.rot / 2), u0[i],
                                 u1[i], a.rot, c[i], n[i]);
            }
            float ss = 0.f, sg = 0.f;
            float v[PPL][16], y[PPL][16];
#pragma unroll
            for (int i = 0; i < PPL; ++i) {
                widen8<F16>(x[i][0], v[i]);
                widen8<F16>(x[i][1], v[i] + 8);
                widen8<F16>(g[i][0], y[i]);
                widen8<F16>(g[i][1], y[i] + 8);
                turn<ADJ, true>(y[i], c[i], n[i]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    ss = fmaf(v[i][e], v[i][e], ss);
                    sg = fmaf(y[i][e] * w[i][e], v[i][e], sg);
                }
            }
            const float rs = rsqrtf(row_sum<LANES>(ss) * (1.f / D) + a.eps);
            // mean(g w xh) with xh = x r
            const float mg = row_sum<LANES>(sg) * rs * (1.f / D);
#pragma unroll
            for (int i = 0; i < PPL; ++i) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float xh = v[i][e] * rs;
                    dw[i][e] = fmaf(y[i][e], xh, dw[i][e]);
                    v[i][e] = rs * (y[i][e] * w[i][e] - xh * mg);
                }
                if (live) {
                    uint16_t* pd = ds + t * dstride + h * D;
                    *reinterpret_cast<uint4*>(pd + 8 * u0[i]) = narrow8<F16>(v[i]);
                    *reinterpret_cast<uint4*>(pd + 8 * u1[i]) = narrow8<F16>(v[i] + 8);
                }
            }
        }
        // the warp's lanes with the same values, then the CTA's warps, in order
#pragma unroll
        for (int i = 0; i < PPL; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float x = dw[i][e];
#pragma unroll
                for (int o = 16; o >= LANES; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (lane < LANES) part[warp][8 * (e < 8 ? u0[i] : u1[i]) + (e & 7)] = x;
            }
        __syncthreads();
        for (int j = threadIdx.x; j < D; j += 32 * kBwdWarps) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < kBwdWarps; ++k) x += part[k][j];
            a.dw_part[((long)kind * gridDim.x + blockIdx.x) * D + j] = x;
        }
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

template <int D, bool F16>
cudaError_t launch_fwd_df(RopeArgs a, cudaStream_t st) {
    using C = RowCfg<D>;
    const int n_rows = a.h_q + a.h_kv + (a.v ? a.h_kv : 0);
    a.segments = cdiv(n_rows, C::ROWS * C::STEPS);
    const long ctas = ((long)a.T * a.segments + kWarps - 1) / kWarps;
    if (a.adjacent) norm_rope_kernel<D, F16, true><<<(unsigned)ctas, 32 * kWarps, 0, st>>>(a);
    else norm_rope_kernel<D, F16, false><<<(unsigned)ctas, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t launch_bwd_df(const RopeArgs& a, int ctas, cudaStream_t st) {
    if (a.adjacent) norm_rope_bwd_kernel<D, F16, true><<<ctas, 32 * kBwdWarps, 0, st>>>(a);
    else norm_rope_bwd_kernel<D, F16, false><<<ctas, 32 * kBwdWarps, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    norm_rope_dw_kernel<<<2 * (D / 32), 1024, 0, st>>>(a, ctas);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a, cudaStream_t st) {
    switch (a.d) {
        case 64: return a.f16 ? launch_fwd_df<64, true>(a, st) : launch_fwd_df<64, false>(a, st);
        case 128: return a.f16 ? launch_fwd_df<128, true>(a, st) : launch_fwd_df<128, false>(a, st);
        case 192: return a.f16 ? launch_fwd_df<192, true>(a, st) : launch_fwd_df<192, false>(a, st);
        case 256: return a.f16 ? launch_fwd_df<256, true>(a, st) : launch_fwd_df<256, false>(a, st);
        default: return cudaErrorInvalidValue;
    }
}

int norm_rope_bwd_ctas(long rows, int d, int sms) {
    const int rows_per_cta = kBwdWarps * (d == 192 ? 8 : 512 / d);
    const long need = (rows + rows_per_cta - 1) / rows_per_cta;
    const long most = (long)sms * 2;
    return (int)(need < 1 ? 1 : need < most ? need : most);
}

cudaError_t launch_norm_rope_bwd(const RopeArgs& a, int ctas, cudaStream_t st) {
    switch (a.d) {
        case 64: return a.f16 ? launch_bwd_df<64, true>(a, ctas, st) : launch_bwd_df<64, false>(a, ctas, st);
        case 128: return a.f16 ? launch_bwd_df<128, true>(a, ctas, st) : launch_bwd_df<128, false>(a, ctas, st);
        case 192: return a.f16 ? launch_bwd_df<192, true>(a, ctas, st) : launch_bwd_df<192, false>(a, ctas, st);
        case 256: return a.f16 ? launch_bwd_df<256, true>(a, ctas, st) : launch_bwd_df<256, false>(a, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
