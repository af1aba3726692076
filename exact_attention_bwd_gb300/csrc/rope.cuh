// What the kernels that normalise and rotate rows of queries and keys share: which values of a row
// a lane holds, and their rotation.
#pragma once
#include "kernels.h"
#include "ptx.cuh"

namespace fa {

constexpr int kUnitBytes = 8192;   // rows of a unit at most (gradient: half of it x, half dy)

template <int D>
struct RowCfg {
    static constexpr int PAIRS = D / 16;               // lanes with values
    static constexpr int LANES = D == 192 ? 16 : PAIRS;  // lanes of a row
    static constexpr int ROWS = 32 / LANES;            // rows of a warp at a time
    // rows of a unit: whole batches of 2 ROWS
    static constexpr int MAX_ROWS = kUnitBytes / (2 * D) / (2 * ROWS) * (2 * ROWS);
};

// The lane's angles from the token's row of the tables: for pairs half the rotated part apart
// c[e], s[e] are those of values 2e, 2e + 1 of unit 0 (and unit 1), e < 4; for adjacent ones
// c[e].x, s[e].x is the angle of the pair e (e < 4 in unit 0, the others in unit 1).  Values
// behind the rotated part get cos 1, sin 0.
template <bool ADJ>
struct Angles {
    float2 c[ADJ ? 8 : 4], s[ADJ ? 8 : 4];
    __device__ __forceinline__ void load(const float* cs, const float* sn, int u0, int u1, int rot) {
        if constexpr (ADJ) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int u = h ? u1 : u0;
                float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (8 * u < rot) {
                    x = *reinterpret_cast<const float4*>(cs + 4 * u);
                    y = *reinterpret_cast<const float4*>(sn + 4 * u);
                }
                c[4 * h] = make_float2(x.x, x.x);
                c[4 * h + 1] = make_float2(x.y, x.y);
                c[4 * h + 2] = make_float2(x.z, x.z);
                c[4 * h + 3] = make_float2(x.w, x.w);
                s[4 * h] = make_float2(-y.x, y.x);
                s[4 * h + 1] = make_float2(-y.y, y.y);
                s[4 * h + 2] = make_float2(-y.z, y.z);
                s[4 * h + 3] = make_float2(-y.w, y.w);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (16 * u0 < rot) {
                    x = *reinterpret_cast<const float4*>(cs + 8 * u0 + 4 * h);
                    y = *reinterpret_cast<const float4*>(sn + 8 * u0 + 4 * h);
                }
                c[2 * h] = make_float2(x.x, x.y);
                c[2 * h + 1] = make_float2(x.z, x.w);
                s[2 * h] = make_float2(y.x, y.y);
                s[2 * h + 1] = make_float2(y.z, y.w);
            }
        }
    }
    // The angles of the inverse.
    __device__ __forceinline__ void turn_round() {
#pragma unroll
        for (int e = 0; e < (ADJ ? 8 : 4); ++e) s[e] = make_float2(-s[e].x, -s[e].y);
    }
    // Turns the lane's 16 values (unit 0 in v[0..3], unit 1 in v[4..7]); BACK: by minus the angle.  Values
    // behind the rotated part are turned by the angle 0, or with STRICT left alone (an infinity
    // times sin 0 would be NaN in its neighbour): unit 0 is rotated if r0, unit 1 if r1.
    template <bool BACK, bool STRICT = false>
    __device__ __forceinline__ void turn(float2* v, bool r0 = true, bool r1 = true) const {
        if constexpr (ADJ) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (STRICT && !(e < 4 ? r0 : r1)) continue;
                const float2 sw = make_float2(v[e].y, v[e].x);
                const float2 ss = BACK ? make_float2(s[e].y, s[e].x) : s[e];
                v[e] = __ffma2_rn(sw, ss, __fmul2_rn(v[e], c[e]));
            }
        } else {
            if (STRICT && !r0) return;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 a = v[e], b = v[e + 4], ns = make_float2(-s[e].x, -s[e].y);
                v[e] = __ffma2_rn(b, BACK ? s[e] : ns, __fmul2_rn(a, c[e]));
                v[e + 4] = __ffma2_rn(a, BACK ? ns : s[e], __fmul2_rn(b, c[e]));
            }
        }
    }
};

// The two units (8 values each, their index in the row) of lane i of a row.
template <int D, bool ADJ>
__device__ __forceinline__ void lane_units(int i, int rot, int& u0, int& u1) {
    const int h = rot >> 4;  // units of half the rotated part
    if (ADJ || i < h) {
        u0 = i;
        u1 = i + (ADJ ? D / 16 : h);
    } else {  // behind the rotated part
        u0 = 2 * i;
        u1 = 2 * i + 1;
    }
}

template <bool F16>
__device__ __forceinline__ void widen8(const uint4& x, float2* v) {
    v[0] = make_float2(lo16<F16>(x.x), hi16<F16>(x.x));
    v[1] = make_float2(lo16<F16>(x.y), hi16<F16>(x.y));
    v[2] = make_float2(lo16<F16>(x.z), hi16<F16>(x.z));
    v[3] = make_float2(lo16<F16>(x.w), hi16<F16>(x.w));
}
template <bool F16>
__device__ __forceinline__ uint4 narrow8(const float2* v) {
    return make_uint4(pack16<F16>(v[0].x, v[0].y), pack16<F16>(v[1].x, v[1].y), pack16<F16>(v[2].x, v[2].y),
                      pack16<F16>(v[3].x, v[3].y));
}

// The lane's 16 weights (null: ones).
template <bool F16>
__device__ __forceinline__ void load_weight(const RopeArgs& a, const void* w, int u0, int u1, float2* v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int u = h ? u1 : u0;
        if (!w) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * h + e] = make_float2(1.f, 1.f);
        } else if (a.weight_f32) {
            const float4* src = reinterpret_cast<const float4*>(w) + 2 * u;
            const float4 x = src[0], y = src[1];
            v[4 * h] = make_float2(x.x, x.y);
            v[4 * h + 1] = make_float2(x.z, x.w);
            v[4 * h + 2] = make_float2(y.x, y.y);
            v[4 * h + 3] = make_float2(y.z, y.w);
        } else {
            widen8<F16>(reinterpret_cast<const uint4*>(w)[u], v + 4 * h);
        }
    }
}

// Sum over the lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

}  // namespace fa
