// stream.h -- weight streaming for few rows: a wavefront multiplies 16 weight rows (output features) with up to
// 16 activation rows (tokens), the weights read straight from global memory into MFMA operands.
//
// With at most 16 tokens a weight byte is used once, so nothing is gained by staging it in LDS: a lane loads
// the 16-byte pieces that its MFMA operand needs (lane l: weight row l % 16, piece l / 16 of every 64 bytes),
// several units of 128 K elements ahead.  The weights are the first MFMA operand, so a result holds
// [feature][token]: lane l has features 4 (l / 16) + r, r = 0..3, of token l % 16.
//
// A unit is 128 elements of K in every weight type: one fp8 scale block, four microscaled groups.
//   fp32 : 8 pieces, v_mfma_f32_16x16x4_f32, four per piece
//   bf16 : 4 pieces, v_mfma_f32_16x16x32_bf16, one per piece
//   fp8  : 2 pieces, one v_mfma_scale_f32_16x16x128_f8f6f4 with unit scales, its result times (activation scale
//          of the row) * (weight block scale) added to the accumulator
//   MXFP4: 1 piece, one v_mfma_scale_f32_16x16x128_f8f6f4 (E2M1 weights, E4M3 activations) that applies both
//          sides' E8M0 scales itself.  Its E4M3 operand holds K 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q +
//          15 on the lanes of group q = l / 16, its E2M1 operand K 32 q .. 32 q + 31, and the scale byte of lane
//          l belongs to K 32 q .. 32 q + 31 of the lane's row.
// Any K order that both operands share gives the same sum, which is all that the other types need.
#pragma once

#include "mx.h"

namespace moe {

enum { ST_F32 = 0, ST_BF16 = 1, ST_FP8 = 2, ST_MX4 = 3 };

template <int ST> struct StreamType;
template <> struct StreamType<ST_F32> { static constexpr int wbytes = 512, abytes = 512; };   // bytes a unit and row
template <> struct StreamType<ST_BF16> { static constexpr int wbytes = 256, abytes = 256; };
template <> struct StreamType<ST_FP8> { static constexpr int wbytes = 128, abytes = 128; };
template <> struct StreamType<ST_MX4> { static constexpr int wbytes = 64, abytes = 128; };

// The lane's pieces of one unit of a weight matrix, with its scales.
template <int ST> struct WUnit {
    static constexpr int N = StreamType<ST>::wbytes / 64;
    i32x4 p[N];
    uint32_t s;                                        // MXFP4: the row's four scale bytes; fp8: block scale bits
    // w: the lane's row + 16 q; ws: MXFP4 the row's scale bytes, fp8 the row block's scales.  Every weight byte is
    // read once by one wavefront: non-temporal.
    __device__ __forceinline__ void load(const uint8_t* w, const uint8_t* ws, int u)
    {
        const uint8_t* b = w + (int64_t)u * StreamType<ST>::wbytes;
#pragma unroll
        for (int j = 0; j < N; j++) p[j] = __builtin_nontemporal_load((const i32x4*)(b + 64 * j));
        if constexpr (ST == ST_FP8 || ST == ST_MX4) s = *(const uint32_t*)(ws + 4 * (int64_t)u);
    }
};

// The lane's pieces of one unit of the activations (row l % 16 of the tile), with their scales.
template <int ST> struct AUnit {
    static constexpr int N = StreamType<ST>::abytes / 64;
    i32x4 p[N];
    uint32_t s;                                        // MXFP4: four scale bytes; fp8: scale bits
    __device__ __forceinline__ void load(const uint8_t* a, const uint8_t* as, int u)
    {
        const uint8_t* b = a + (int64_t)u * StreamType<ST>::abytes;
#pragma unroll
        for (int j = 0; j < N; j++) p[j] = *(const i32x4*)(b + 64 * j);
        if constexpr (ST == ST_FP8 || ST == ST_MX4) s = *(const uint32_t*)(as + 4 * (int64_t)u);
    }
};

// acc += W unit . A unit; q = lane / 16.
template <int ST> __device__ __forceinline__ void stream_mma(f32x4& acc, const WUnit<ST>& w, const AUnit<ST>& a, int q)
{
    if constexpr (ST == ST_F32) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const f32x4 wf = __builtin_bit_cast(f32x4, w.p[j]), af = __builtin_bit_cast(f32x4, a.p[j]);
#pragma unroll
            for (int e = 0; e < 4; e++) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[e], af[e], acc, 0, 0, 0);
        }
    } else if constexpr (ST == ST_BF16) {
#pragma unroll
        for (int j = 0; j < 4; j++)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.p[j]),
                                                          __builtin_bit_cast(bf16x8, a.p[j]), acc, 0, 0, 0);
    } else if constexpr (ST == ST_FP8) {
        const i32x8 wv = {w.p[0].x, w.p[0].y, w.p[0].z, w.p[0].w, w.p[1].x, w.p[1].y, w.p[1].z, w.p[1].w};
        const i32x8 av = {a.p[0].x, a.p[0].y, a.p[0].z, a.p[0].w, a.p[1].x, a.p[1].y, a.p[1].z, a.p[1].w};
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, zero, 0, 0, 0, 127, 0, 127);
        const float s = __uint_as_float(w.s) * __uint_as_float(a.s);
#pragma unroll
        for (int r = 0; r < 4; r++) acc[r] += p[r] * s;
    } else {
        const i32x8 wv = {w.p[0].x, w.p[0].y, w.p[0].z, w.p[0].w, 0, 0, 0, 0};
        const i32x8 av = {a.p[0].x, a.p[0].y, a.p[0].z, a.p[0].w, a.p[1].x, a.p[1].y, a.p[1].z, a.p[1].w};
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, acc, 4, 0, 0, (int)(w.s >> (8 * q)), 0,
                                                               (int)(a.s >> (8 * q)));
    }
}

// acc1 += W1 . A, and for UP acc3 += W3 . A, over the units [u0, u1), D units in flight.  Pointers as in load();
// past the end the last unit is loaded again (a cache hit), so no load stands behind a branch.
template <int ST, bool UP, int D>
__device__ __forceinline__ void stream_units(f32x4& acc1, f32x4& acc3, const uint8_t* w1, const uint8_t* w1s,
                                             const uint8_t* w3, const uint8_t* w3s, const uint8_t* a, const uint8_t* as,
                                             int u0, int u1, int q)
{
    if (u0 >= u1) return;
    WUnit<ST> r1[D], r3[UP ? D : 1];
    AUnit<ST> ra[D];
    auto load = [&](int j, int u) {
        r1[j].load(w1, w1s, u);
        if constexpr (UP) r3[j].load(w3, w3s, u);
        ra[j].load(a, as, u);
    };
#pragma unroll
    for (int j = 0; j < D; j++) load(j, min(u0 + j, u1 - 1));
    for (int u = u0; u < u1; u += D) {
#pragma unroll
        for (int j = 0; j < D; j++) {
            if (u + j < u1) {
                stream_mma<ST>(acc1, r1[j], ra[j], q);
                if constexpr (UP) stream_mma<ST>(acc3, r3[j], ra[j], q);
            }
            load(j, min(u + j + D, u1 - 1));
        }
    }
}

}  // namespace moe
