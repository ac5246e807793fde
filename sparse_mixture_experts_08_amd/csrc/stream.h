// stream.h -- weight streaming for few rows: a wavefront multiplies 16 weight rows (output features) with up to
// 16 activation rows (tokens).
//
// With at most 16 tokens a weight byte is used once, and the loads decide the time.  HBM gives the most where one
// load instruction takes whole 128-byte lines of a few rows with the non-temporal hint: a copyless read of 4 GB in
// rows of 3.5 to 14 KB runs at 7.0 to 7.15 TB/s with 8 rows x 128 bytes an instruction, at 6.0 to 6.3 without the
// hint, and at 5.0 to 5.3 with the hint and the 16 rows x 64 bytes that an MFMA operand would take as they are
// (lane l: row l % 16, bytes 16 (l / 16)).  So a lane loads 16 bytes of row l / 8, and a line pair of 16 rows
// changes hands through 2 KB of LDS of the wavefront's own: no barrier, since a wavefront's LDS accesses are done
// in order.  The weights are the first MFMA operand, so a result holds [feature][token]: lane l has features
// 4 (l / 16) + r, r = 0..3, of token l % 16.
//
// A unit is one 128-byte line of every weight row:
//   fp32 :  32 elements of K, v_mfma_f32_16x16x4_f32, eight per unit
//   bf16 :  64, v_mfma_f32_16x16x32_bf16, two per unit
//   fp8  : 128, one v_mfma_scale_f32_16x16x128_f8f6f4 with unit scales, its result times (activation scale of the
//          row) * (weight block scale) added to the accumulator
//   MXFP4: 256, two v_mfma_scale_f32_16x16x128_f8f6f4 (E2M1 weights, E4M3 activations) that apply both sides' E8M0
//          scales themselves.  The E4M3 operand holds K 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15 on the
//          lanes of group q = l / 16, the E2M1 operand K 32 q .. 32 q + 31, and the scale byte of lane l belongs to
//          K 32 q .. 32 q + 31 of the lane's row.  K is a multiple of 128, so a row may end in half a unit.
// Any K order that both operands share gives the same sum, which is all that the other types need.
#pragma once

#include "mx.h"

namespace moe {

enum { ST_F32 = 0, ST_BF16 = 1, ST_FP8 = 2, ST_MX4 = 3 };

// K elements of a unit; 16-byte pieces of activations that a lane holds of it (64 bytes apart in the row).
template <int ST> struct StreamType;
template <> struct StreamType<ST_F32> { static constexpr int K = 32, NA = 2; };
template <> struct StreamType<ST_BF16> { static constexpr int K = 64, NA = 2; };
template <> struct StreamType<ST_FP8> { static constexpr int K = 128, NA = 2; };
template <> struct StreamType<ST_MX4> { static constexpr int K = 256, NA = 4; };

constexpr int STREAM_TILE = 16 * 128;                  // LDS bytes of one unit

template <int ST> __device__ __forceinline__ int stream_units_of(int K)
{
    return (K + StreamType<ST>::K - 1) / StreamType<ST>::K;
}

// Where a wavefront's 16 weight rows lie: rows 0-7 from p0 and rows 8-15 from p1 (wavefront-uniform), each lane's
// offset in them, and the lane's own scale pointer.
struct WRows {
    const uint8_t *p0, *p1;
    uint32_t off;                                      // row l / 8, 16-byte chunk l % 8
    int half;                                          // MXFP4: the unit that is only half there, or -1
    uint32_t offh;                                     // ... and the offset for it: chunks 4 .. 7 read 0 .. 3 again
    const uint8_t* s;                                  // MXFP4: scale bytes of row l % 16; fp8: its block row's floats
};

// ld: bytes between rows; K: the rows' length.
template <int ST>
__device__ __forceinline__ WRows weight_rows(const uint8_t* p0, const uint8_t* p1, const uint8_t* s, int64_t ld, int K, int lane)
{
    const uint32_t row = (lane >> 3) * (uint32_t)ld;
    return {p0, p1, row + (lane & 7) * 16, ST == ST_MX4 && K % 256 ? K / 256 : -1, row + (lane & 3) * 16, s};
}

// The lane's part of one unit of weights on its way, with its scales.
template <int ST> struct WUnit {
    i32x4 p[2];                                        // rows l / 8 and 8 + l / 8
    uint32_t s[ST == ST_MX4 ? 2 : 1];                  // MXFP4: row l % 16's scale bytes, 128 elements each; fp8: scale bits
    // The next unit of r, and r moved on by n units (0 or 1); h: the unit is only half there.
    __device__ __forceinline__ void load(WRows& r, bool h, int n)
    {
        const uint32_t o = ST == ST_MX4 && h ? r.offh : r.off;
        p[0] = __builtin_nontemporal_load((const i32x4*)(r.p0 + o));
        p[1] = __builtin_nontemporal_load((const i32x4*)(r.p1 + o));
        r.p0 += 128 * n;
        r.p1 += 128 * n;
        if constexpr (ST == ST_FP8) {
            s[0] = *(const uint32_t*)r.s;
            r.s += 4 * n;
        }
        if constexpr (ST == ST_MX4) {
            s[0] = ((const uint32_t*)r.s)[0];
            s[1] = ((const uint32_t*)r.s)[h ? 0 : 1];
            r.s += 8 * n;
        }
    }
    // Into the wavefront's tile: chunk c of row r at chunk c ^ f(r), f(r) = (r ^ (r >> 3 & 1)) & 7, so that the 16
    // rows of a read fall on distinct banks.
    __device__ __forceinline__ void put(uint8_t* tile, int lane) const
    {
        const int row = lane >> 3, c = lane & 7;
        *(i32x4*)(tile + row * 128 + ((c ^ row) << 4)) = p[0];
        *(i32x4*)(tile + (row + 8) * 128 + ((c ^ (row ^ 1)) << 4)) = p[1];
    }
    // The pieces of row l % 16 as an MFMA operand takes them: chunks q and 4 + q.
    static __device__ __forceinline__ void get(const uint8_t* tile, int lane, i32x4 (&v)[2])
    {
        const int row = lane & 15, q = lane >> 4, f = (row ^ (row >> 3)) & 7;
        v[0] = *(const i32x4*)(tile + row * 128 + ((q ^ f) << 4));
        v[1] = *(const i32x4*)(tile + row * 128 + (((4 + q) ^ f) << 4));
    }
};

// Activation rows: lane l's row (l % 16 of the tile) at p + off, its scales at s + soff.
struct ARows {
    const uint8_t *p, *s;
    uint32_t off, soff;                                // off includes 16 q
    int half;
};

template <int ST> struct AUnit {
    i32x4 p[StreamType<ST>::NA];
    uint32_t s[ST == ST_MX4 ? 2 : 1];
    __device__ __forceinline__ void load(const ARows& r, int u)
    {
        const uint8_t* b = r.p + (int64_t)u * 64 * StreamType<ST>::NA;
        const bool h = ST == ST_MX4 && u == r.half;
#pragma unroll
        for (int j = 0; j < StreamType<ST>::NA; j++) p[j] = *(const i32x4*)(b + (j >= 2 && h ? j - 2 : j) * 64 + r.off);
        if constexpr (ST == ST_FP8) s[0] = *(const uint32_t*)(r.s + (int64_t)u * 4 + r.soff);
        if constexpr (ST == ST_MX4) {
            const uint8_t* c = r.s + (int64_t)u * 8;
            s[0] = *(const uint32_t*)(c + r.soff);
            s[1] = *(const uint32_t*)(c + (h ? 0 : 4) + r.soff);
        }
    }
};

// acc += W unit . A unit, w the operand pieces, ws the scales; whole: both halves of an MXFP4 unit; q = lane / 16.
template <int ST>
__device__ __forceinline__ void stream_mma(f32x4& acc, const i32x4 (&w)[2], const uint32_t* ws, const AUnit<ST>& a, bool whole, int q)
{
    if constexpr (ST == ST_F32) {
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const f32x4 wf = __builtin_bit_cast(f32x4, w[j]), af = __builtin_bit_cast(f32x4, a.p[j]);
#pragma unroll
            for (int e = 0; e < 4; e++) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[e], af[e], acc, 0, 0, 0);
        }
    } else if constexpr (ST == ST_BF16) {
#pragma unroll
        for (int j = 0; j < 2; j++)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[j]),
                                                          __builtin_bit_cast(bf16x8, a.p[j]), acc, 0, 0, 0);
    } else if constexpr (ST == ST_FP8) {
        const i32x8 wv = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
        const i32x8 av = {a.p[0].x, a.p[0].y, a.p[0].z, a.p[0].w, a.p[1].x, a.p[1].y, a.p[1].z, a.p[1].w};
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, zero, 0, 0, 0, 127, 0, 127);
        const float s = __uint_as_float(ws[0]) * __uint_as_float(a.s[0]);
#pragma unroll
        for (int r = 0; r < 4; r++) acc[r] += p[r] * s;
    } else {
#pragma unroll
        for (int j = 0; j < 2; j++) {
            if (j == 1 && !whole) break;
            const i32x8 wv = {w[j].x, w[j].y, w[j].z, w[j].w, 0, 0, 0, 0};
            const i32x4 lo = a.p[2 * j], hi = a.p[2 * j + 1];
            const i32x8 av = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, acc, 4, 0, 0, (int)(ws[j] >> (8 * q)), 0,
                                                                   (int)(a.s[j] >> (8 * q)));
        }
    }
}

// acc += W . A with D weight units in flight.  tile: the wavefront's own LDS.  A_LDS: the activations lie in LDS and
// are read as they are needed; otherwise their units travel with the weights'.  (Vector loads come back in order, so
// the wait for an activation load that was issued later than far-ahead weight loads would be a wait for those.)
// The scheduling barriers keep the loads in the order of their
// units, in the prologue as in the loop: a unit's wait then leaves the D - 1 units behind it in flight.  (Without
// them the compiler orders the prologue its own way, and the loop's waits, which have to hold for both, drain almost
// every load.)
template <int ST, bool A_LDS, int D> struct Stream {
    WUnit<ST> w[D];
    AUnit<ST> a[A_LDS ? 1 : D];
    WRows wr;                                          // from the next unit to load on
    int next;

    __device__ __forceinline__ void load(int j, const ARows& ar, int n = 1)
    {
        w[j].load(wr, next == wr.half, n);
        if constexpr (!A_LDS) a[j].load(ar, next);
        next += n;
        __builtin_amdgcn_sched_barrier(0);
    }
    // The first units of nu; of fewer than D, the last one again.
    __device__ __forceinline__ void begin(const WRows& r, const ARows& ar, int nu)
    {
        wr = r;
        next = 0;
#pragma unroll
        for (int j = 0; j < D; j++)
            load(j, ar, j + 1 < nu || j == D - 1);
    }
    __device__ __forceinline__ void mma(int j, f32x4& acc, const ARows& ar, int u, int ua, uint8_t* tile, int lane)
    {
        i32x4 f[2];
        w[j].put(tile, lane);
        if constexpr (A_LDS) {
            AUnit<ST> al;
            al.load(ar, ua);
            WUnit<ST>::get(tile, lane, f);
            stream_mma<ST>(acc, f, w[j].s, al, u != wr.half, lane >> 4);
        } else {
            WUnit<ST>::get(tile, lane, f);
            stream_mma<ST>(acc, f, w[j].s, a[j], u != wr.half, lane >> 4);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // Units [u0, u1) of nu, u0 a multiple of D; in LDS ar counts its units from u0.  The rounds whose every unit has
    // a successor to load run in a loop without a branch; the last two rounds stand by themselves, so that nothing
    // past the end is loaded.
    __device__ __forceinline__ void run(f32x4& acc, const ARows& ar, int u0, int u1, int nu, uint8_t* tile, int lane)
    {
        int u = u0;
        for (; u < u1 && u + 2 * D <= nu; u += D) {
#pragma unroll
            for (int j = 0; j < D; j++) {
                mma(j, acc, ar, u + j, u + j - u0, tile, lane);
                load(j, ar);
            }
        }
        if (u < u1 && u + D <= nu) {
#pragma unroll
            for (int j = 0; j < D; j++) {
                mma(j, acc, ar, u + j, u + j - u0, tile, lane);
                if (u + j + D < nu) load(j, ar);
            }
            u += D;
        }
        if (u < u1) {
#pragma unroll
            for (int j = 0; j < D; j++)
                if (u + j < u1) mma(j, acc, ar, u + j, u + j - u0, tile, lane);
        }
    }
};

}  // namespace moe
