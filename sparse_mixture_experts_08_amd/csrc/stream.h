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
constexpr int STREAM_PAD = 32;                         // behind a row of activations in LDS: see WUnit::put

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
    int ns;                                            // 4-byte words there
};

// A pointer that is the same in every lane, as a scalar.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p)
{
    const uint64_t v = (uint64_t)p;
    return (const uint8_t*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                            (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// ld: bytes between rows; K: the rows' length.
template <int ST>
__device__ __forceinline__ WRows weight_rows(const uint8_t* p0, const uint8_t* p1, const uint8_t* s, int64_t ld, int K, int lane)
{
    const uint32_t row = (lane >> 3) * (uint32_t)ld;
    return {uniform(p0), uniform(p1), row + (lane & 7) * 16, ST == ST_MX4 && K % 256 ? K / 256 : -1, row + (lane & 3) * 16, s, K / 128};
}

// The lane's part of one unit of weights on its way.
template <int ST> struct WUnit {
    i32x4 p[2];                                        // rows l / 8 and 8 + l / 8
    __device__ __forceinline__ void load(const WRows& r, int u)
    {
        const uint32_t o = ST == ST_MX4 && u == r.half ? r.offh : r.off;
        p[0] = __builtin_nontemporal_load((const i32x4*)(r.p0 + (int64_t)u * 128 + o));
        p[1] = __builtin_nontemporal_load((const i32x4*)(r.p1 + (int64_t)u * 128 + o));
    }
    // Into the wavefront's tile: chunk c of row r at chunk c ^ (r / 2 % 8).  A 16-byte read takes 16 lanes a clock: lanes
    // 0-3, 12-15 and 20-27, then 4-11, 16-19 and 28-31, and so on, that is half of the 16 rows at one chunk and the
    // other half at the next, which this places on all 64 banks.
    __device__ __forceinline__ void put(uint8_t* tile, int lane) const
    {
        const int row = lane >> 3, c = lane & 7;
        *(i32x4*)(tile + row * 128 + ((c ^ row >> 1) << 4)) = p[0];
        *(i32x4*)(tile + (row + 8) * 128 + ((c ^ (row >> 1 ^ 4)) << 4)) = p[1];
    }
    // The pieces of row l % 16 as an MFMA operand takes them: chunks q and 4 + q.
    static __device__ __forceinline__ void get(const uint8_t* tile, int lane, i32x4 (&v)[2])
    {
        const int row = lane & 15, q = lane >> 4, f = row >> 1;
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
            if (h) p[2] = p[3] = (i32x4){0, 0, 0, 0};  // the half that is not there
        }
    }
};

// acc += W unit . A unit, w the operand pieces, ws the scales (MXFP4: one word a half); q = lane / 16.
template <int ST>
__device__ __forceinline__ void stream_mma(f32x4& acc, const i32x4 (&w)[2], const uint32_t (&ws)[2], const AUnit<ST>& a, int q)
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
            const i32x8 wv = {w[j].x, w[j].y, w[j].z, w[j].w, 0, 0, 0, 0};
            const i32x4 lo = a.p[2 * j], hi = a.p[2 * j + 1];
            const i32x8 av = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, acc, 4, 0, 0, (int)(ws[j] >> (8 * q)), 0,
                                                                   (int)(a.s[j] >> (8 * q)));
        }
    }
}

// A stream of weight units through registers, D in flight, one matrix after the other.  fill() issues the first D
// units; a round multiplies D units and, with MORE, issues the D after them in their places: a matrix's rounds are
// all alike, and before its last one start() may name the matrix that follows, so that the loads never pause.  Past
// a matrix's end its last unit is loaded again (nu need not be a multiple of D); nothing is multiplied there.
// tile: the wavefront's own LDS.  A_LDS: the activations lie in LDS and are read as they are needed; otherwise their
// units travel with the weights'.  (Vector loads come back in order, so the wait for an activation load that was
// issued later than far-ahead weight loads would be a wait for those.)  Scales: one word load a lane brings the words
// of several units (MXFP4: two units, the word 2 u + q of row l % 16 to lane l; fp8: four units, the word u + l % 4 of
// the lane's block row), handed around by lane permutes; as a load per unit and half they would be as many line
// requests as the weights.  The scheduling barriers keep the loads in the order of their units, with no branch around
// them: a unit's wait then leaves the D - 1 units behind it in flight.  (Left alone, the compiler orders the first
// loads its own way, and the waits, which have to hold for them too, drain almost every load.)
template <int ST, bool A_LDS, int D> struct Stream {
    static constexpr int SU = ST == ST_MX4 ? 2 : ST == ST_FP8 ? 4 : 1;         // units a scale load serves
    static_assert(D % SU == 0, "whole scale loads a round");
    WUnit<ST> w[D];
    uint32_t s[D / SU];
    AUnit<ST> a[A_LDS ? 1 : D];
    WRows wr;
    ARows ar;                                          // !A_LDS: the activations that travel along, and whether they
    int ar_step = 1;                                   // advance (0: the first unit again and again, unused)
    int next, end;                                     // the unit to load next, and the first past those to load

    // Units [u0, u1) of these rows come next; u0 a multiple of SU.  (None: unit u0, if there is one, unused.)
    __device__ __forceinline__ void start(const WRows& r, int u0, int u1)
    {
        wr = r;
        next = u0;
        end = u1;
    }
    __device__ __forceinline__ void stay() { end = 1; }
    __device__ __forceinline__ void load(int j, int lane)
    {
        const int u = max(min(next, end - 1), 0);
        w[j].load(wr, u);
        if constexpr (ST == ST_MX4 || ST == ST_FP8) {
            if (j % SU == SU - 1) {                    // behind the last of the units it serves: the old words are used up
                const int first = next - (SU - 1), i = ST == ST_MX4 ? 2 * first + (lane >> 4) : first + (lane & 3);
                s[j / SU] = ((const uint32_t*)wr.s)[max(min(i, wr.ns - 1), 0)];
            }
        }
        if constexpr (!A_LDS) a[j].load(ar, u * ar_step);
        next++;
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void fill(int lane)
    {
#pragma unroll
        for (int j = 0; j < D; j++) load(j, lane);
    }
    // acc += units u .. u + D - 1, of those below u1.  al: activations, if they lie in LDS (LDS: in any case), their
    // units counted from ua.
    template <bool MORE, bool LDS = A_LDS>
    __device__ __forceinline__ void round(f32x4& acc, const ARows& al, int u, int u1, int ua, uint8_t* tile, int lane)
    {
#pragma unroll
        for (int j = 0; j < D; j++) {
            if (u + j < u1) {
                i32x4 f[2];
                uint32_t ws[2] = {0, 0};
                w[j].put(tile, lane);
                if constexpr (ST == ST_MX4) {          // words 2 j, 2 j + 1 of the four that the row's lanes hold
                    ws[0] = __shfl(s[j / 2], (lane & 15) + 32 * (j % 2), 64);
                    ws[1] = __shfl(s[j / 2], (lane & 15) + 32 * (j % 2) + 16, 64);
                } else if constexpr (ST == ST_FP8) {
                    ws[0] = __shfl(s[j / 4], (lane & 60) + j % 4, 64);
                }
                if constexpr (LDS) {
                    AUnit<ST> x;
                    x.load(al, u + j - ua);
                    WUnit<ST>::get(tile, lane, f);
                    stream_mma<ST>(acc, f, ws, x, lane >> 4);
                } else {
                    WUnit<ST>::get(tile, lane, f);
                    stream_mma<ST>(acc, f, ws, a[j], lane >> 4);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (MORE) load(j, lane);
        }
    }
};

}  // namespace moe
