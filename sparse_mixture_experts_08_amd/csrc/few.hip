// few.hip -- the whole layer for at most MOE_FEW_MAX_T tokens in two launches (moe_forward_few).
//
// With so few tokens every weight byte is read once and used for a handful of multiplications: the weights of
// the selected experts bound the layer, and at one token also whatever keeps HBM idle, which is each launch's
// start and drain and each serial step in between.  So:
//   launch 1 (few_prepare_kernel): router logits, one block per expert; the activations' quantisation, where the
//     weight type has one; the counters of launch 2 set to zero.
//   launch 2 (few_layer_kernel): a grid that fills the card once, whose blocks take work items from one counter
//     until none is left.  Every block first selects the experts itself (a top-k over T rows of logits, cheaper
//     than a hand-off between blocks).  Items, in this order: the up products of the shared expert and of each
//     selected expert, 16 hidden features an item; then their down products, 128 output features an item.  A
//     down item waits for its expert's up items, and the block that completes the last down item of a column
//     range sums the experts' outputs there.  No launch boundary lies between the phases: blocks stream down
//     weights while others finish up items.
//
// Why every wait ends.  Blocks take item numbers from the counter in ascending order, and an item waits only for
// items of lower numbers.  Take the lowest unfinished item: the block that holds it is running (it took the
// number) and has finished what it held before, since that has a lower number; what the item waits for is
// finished too; so it completes.  This holds for any number of resident blocks, in any order of dispatch, and
// beside other kernels (a second call of this one among them).
//
// Router logits.  The products x[t][i] * Wg[e][i] are exact in fp64 and are summed there, the bias is added, and
// the sum is rounded once to fp32: over a row of 2^13 terms fp64's error is below 2^-40 of the terms' magnitudes,
// so the logit is the correctly rounded one but for ties at 2^-17 of an fp32 step.  The order of a sum then does
// not matter, and the row can be split over a block (the FMA chain of moe_route takes 7168 dependent steps).
#include <type_traits>

#include "gemm.h"
#include "stream.h"
#include "topk.h"

namespace moe {

constexpr int FEW_T = MOE_FEW_MAX_T;
constexpr int FEW_SLOTS = FEW_T * 16;                  // (token, slot) pairs at most
constexpr int FEW_GROUPS = FEW_SLOTS + 1;              // selected experts and the shared one, at most
constexpr int FEW_NW = 8;                              // wavefronts per block of launch 2
constexpr int FEW_UP = 16;                             // hidden features per up item
constexpr int FEW_DN = 16 * FEW_NW;                    // output features per down item

struct FewArgs {
    int T, d, E, k, inter, inter_s, inter_max;
    const uint8_t* x;                                  // [T, d] act dtype, or codes
    const uint8_t* xs;                                 // scales of x (fp8: fp32; MXFP4: E8M0)
    const float* logits;                               // [T, E]
    const uint8_t *W1, *W3, *W2, *W1s, *W3s, *W2s;
    const uint8_t *S1, *S3, *S2, *S1s, *S3s, *S2s;
    uint8_t* h;                                        // [T k + T, inter_max] act dtype
    uint8_t* y_rows;                                   // [T k + T, d] act dtype
    uint8_t* y;
    int32_t *idx_out, *w_out_bits, *counts_out;        // optional
    int32_t *ticket, *up_done, *col_done;              // counters: [1], [FEW_GROUPS], [d / FEW_DN]
};

// ---------------------------------------------------------------------------------------------------
// Launch 1.  Blocks [0, E): the logits of one expert for every token.  Blocks [E, E + nq): quantisation of x.
// The last block clears the counters.
// ---------------------------------------------------------------------------------------------------
template <typename XT> __device__ __forceinline__ void load4(const XT* p, double (&v)[4]);
template <> __device__ __forceinline__ void load4<uint16_t>(const uint16_t* p, double (&v)[4])
{
    const uint2 r = *(const uint2*)p;
    v[0] = (double)__uint_as_float(r.x << 16);
    v[1] = (double)__uint_as_float(r.x & 0xFFFF0000u);
    v[2] = (double)__uint_as_float(r.y << 16);
    v[3] = (double)__uint_as_float(r.y & 0xFFFF0000u);
}
template <> __device__ __forceinline__ void load4<float>(const float* p, double (&v)[4])
{
    const float4 r = *(const float4*)p;
    v[0] = (double)r.x; v[1] = (double)r.y; v[2] = (double)r.z; v[3] = (double)r.w;
}

template <int ST, int TM>
__global__ __launch_bounds__(256) void few_prepare_kernel(const void* __restrict__ xv, const float* __restrict__ Wg,
                                                          const float* __restrict__ bias, float* __restrict__ logits,
                                                          int T, int d, int E, uint8_t* __restrict__ xq,
                                                          uint8_t* __restrict__ xs, int32_t* __restrict__ counters,
                                                          int n_counters)
{
    typedef typename std::conditional<ST == ST_F32, float, uint16_t>::type XT;
    const XT* x = (const XT*)xv;
    const int tid = threadIdx.x, b = blockIdx.x;
    if (b < E) {
        __shared__ double part[4][TM];
        double acc[TM];
#pragma unroll
        for (int t = 0; t < TM; t++) acc[t] = 0.0;
        const float* wrow = Wg + (size_t)b * d;
        for (int i = tid * 4; i < d; i += 1024) {
            double w[4];
            load4<float>(wrow + i, w);
#pragma unroll
            for (int t = 0; t < TM; t++) {
                double v[4];
                load4<XT>(x + (size_t)min(t, T - 1) * d + i, v);
#pragma unroll
                for (int e = 0; e < 4; e++) acc[t] = __builtin_fma(v[e], w[e], acc[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < TM; t++) {
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1) acc[t] += __shfl_xor(acc[t], off, 64);
            if ((tid & 63) == 0) part[tid >> 6][t] = acc[t];
        }
        __syncthreads();
        if (tid < T) {
            double s = ((part[0][tid] + part[1][tid]) + part[2][tid]) + part[3][tid];
            if (bias) s += (double)bias[b];
            logits[(size_t)tid * E + b] = (float)s;
        }
        return;
    }
    if (b == (int)gridDim.x - 1) {
        for (int i = tid; i < n_counters; i += 256) counters[i] = 0;
        return;
    }
    if constexpr (ST == ST_MX4) {
        const int64_t i = (int64_t)(b - E) * 256 + tid;               // eight elements each
        if (i >= (int64_t)T * d / 8) return;                           // whole groups of 16 lanes leave together
        float v[8];
        bf16x8_to_f32(((const uint4*)x)[i], v);
        const uint32_t c = mx_scale_code<false>(quad_max(mx_amax8(v)));
        ((uint2*)xq)[i] = c == 255u ? make_uint2(0u, 0u) : mx_pack_fp8(v, c);
        if ((i & 3) == 0) xs[i >> 2] = (uint8_t)c;
    } else if constexpr (ST == ST_FP8) {
        const int64_t i = (int64_t)(b - E) * 256 + tid;
        if (i >= (int64_t)T * d / 8) return;
        float v[8];
        bf16x8_to_f32(((const uint4*)x)[i], v);
        float sc;
        ((uint2*)xq)[i] = quant8_e4m3(v, sc);
        if ((i & 15) == 0) ((float*)xs)[i >> 4] = sc;
    }
}

// ---------------------------------------------------------------------------------------------------
// Launch 2.
// ---------------------------------------------------------------------------------------------------
template <int ST> struct FewH;                         // the chunk of h that a down item keeps in LDS
template <> struct FewH<ST_F32> { static constexpr int KC = 512, row = KC * 4; };
template <> struct FewH<ST_BF16> { static constexpr int KC = 1024, row = KC * 2; };
template <> struct FewH<ST_FP8> { static constexpr int KC = 2048, row = KC; };
template <> struct FewH<ST_MX4> { static constexpr int KC = 2048, row = KC; };

__device__ __forceinline__ int32_t take(int32_t* counter)
{
    return __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int ST>
__global__ __launch_bounds__(64 * FEW_NW) void few_layer_kernel(FewArgs a)
{
    constexpr bool BF = ST != ST_F32;                  // activations are bf16
    constexpr int AB = BF ? 2 : 4, NT = 64 * FEW_NW;
    constexpr int KC = FewH<ST>::KC, HSTR = FewH<ST>::row + 16;
    constexpr int DU = ST == ST_MX4 ? 4 : ST == ST_FP8 ? 3 : 2, DD = ST == ST_MX4 ? 8 : ST == ST_FP8 ? 4 : 2;
    constexpr int RED = FEW_NW * 2 * 256 * 4, HB = 16 * HSTR;
    typedef StreamType<ST> TY;
    __shared__ __attribute__((aligned(16))) uint8_t buf[RED > HB ? RED : HB];   // up: partial sums; down: h
    __shared__ __attribute__((aligned(16))) uint8_t hsc[16 * (KC / 32)];        // down: scales of the h chunk
    __shared__ int s_idx[FEW_SLOTS];                   // expert of each slot
    __shared__ float s_w[FEW_SLOTS];
    __shared__ uint16_t s_order[FEW_SLOTS];            // a token's slots by ascending expert
    __shared__ uint32_t s_tok[1024];                   // tokens (bits) of each expert
    __shared__ uint16_t s_grp[1024];                   // group of each selected expert
    __shared__ uint16_t s_exp[FEW_GROUPS], s_n[FEW_GROUPS];
    __shared__ uint16_t s_slot[FEW_GROUPS][16];        // the slots of a group's rows (group 0: tokens)
    __shared__ int scan[FEW_NW + 1];
    __shared__ int s_item, s_last;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r16 = lane & 15, q = lane >> 4;
    const int T = a.T, k = a.k, E = a.E, d = a.d, slots = T * k;

    // ---- selection: every block for itself
    for (int e = tid; e < 1024; e += NT) s_tok[e] = 0;
    __syncthreads();
    if (E <= 256) {
        if (wave * 4 < T) {                            // wavefront-uniform
            const int t = wave * 4 + q;
            int e;
            float w;
            topk_group<16, 16>(a.logits + (size_t)min(t, T - 1) * E, nullptr, E, k, r16, e, w);
            if (t < T && r16 < k) {
                s_idx[t * k + r16] = e;
                s_w[t * k + r16] = w;
                atomicOr(&s_tok[e], 1u << t);
            }
        }
    } else {
        for (int t = wave; t < T; t += FEW_NW) {
            int e;
            float w;
            topk_group<64, 16>(a.logits + (size_t)t * E, nullptr, E, k, lane, e, w);
            if (lane < k) {
                s_idx[t * k + lane] = e;
                s_w[t * k + lane] = w;
                atomicOr(&s_tok[e], 1u << t);
            }
        }
    }
    __syncthreads();
    const uint32_t m0 = s_tok[2 * tid], m1 = s_tok[2 * tid + 1];
    int n_sel;
    const int rank = block_exclusive_scan<NT>((m0 != 0) + (m1 != 0), &n_sel, scan);
    if (m0) {
        s_grp[2 * tid] = (uint16_t)(1 + rank);
        s_exp[1 + rank] = (uint16_t)(2 * tid);
        s_n[1 + rank] = (uint16_t)__popc(m0);
    }
    if (m1) {
        const int r = 1 + rank + (m0 != 0);
        s_grp[2 * tid + 1] = (uint16_t)r;
        s_exp[r] = (uint16_t)(2 * tid + 1);
        s_n[r] = (uint16_t)__popc(m1);
    }
    if (tid < 16) s_slot[0][tid] = (uint16_t)(slots + min(tid, T - 1));
    if (tid == 0) s_n[0] = (uint16_t)T;
    __syncthreads();
    if (tid < slots) {
        const int t = tid / k, e = s_idx[tid];
        s_slot[s_grp[e]][__popc(s_tok[e] & ((1u << t) - 1u))] = (uint16_t)tid;
        int before = 0;
        for (int j = 0; j < k; j++) before += s_idx[t * k + j] < e;
        s_order[t * k + before] = (uint16_t)tid;
    }
    if (blockIdx.x == 0) {
        if (tid < slots) {
            if (a.idx_out) a.idx_out[tid] = s_idx[tid];
            if (a.w_out_bits) a.w_out_bits[tid] = __float_as_int(s_w[tid]);
        }
        if (a.counts_out)
            for (int e = tid; e < E; e += NT) a.counts_out[e] = __popc(s_tok[e]);
    }
    __syncthreads();

    // ---- items
    const int ng = 1 + n_sel, nu_s = a.inter_s / FEW_UP, nu_r = a.inter / FEW_UP, ncol = d / FEW_DN;
    const int n_up = nu_s + n_sel * nu_r, total = n_up + ng * ncol;
    int next = 0;
    if (tid == 0) next = take(a.ticket);
    for (;;) {
        if (tid == 0) s_item = next;
        __syncthreads();
        const int item = s_item;
        if (item >= total) break;                      // every block comes to a number past the end
        if (tid == 0) next = take(a.ticket);           // in flight during the item

        if (item < n_up) {
            // ---- 16 hidden features of one expert: eight wavefronts share K, partial sums joined through LDS
            const int g = item < nu_s ? 0 : 1 + (item - nu_s) / nu_r;
            const int f0 = (item < nu_s ? item : (item - nu_s) % nu_r) * FEW_UP;
            const bool shared = g == 0;
            const int e = shared ? 0 : s_exp[g], n = s_n[g];
            const int slot = s_slot[g][r16 < n ? r16 : 0];             // lanes past the rows repeat the first
            const int64_t tok = slot < slots ? slot / k : slot - slots;
            const int64_t ldw = (int64_t)(d / 128) * TY::wbytes;
            const int64_t wrow = (shared ? 0 : (int64_t)e * a.inter) + f0 + r16;
            const uint8_t* w1 = (shared ? a.S1 : a.W1) + wrow * ldw + 16 * q;
            const uint8_t* w3 = (shared ? a.S3 : a.W3) + wrow * ldw + 16 * q;
            const uint8_t *w1s = nullptr, *w3s = nullptr, *as = nullptr;
            if constexpr (ST == ST_MX4) {
                w1s = (shared ? a.S1s : a.W1s) + wrow * (d / 32);
                w3s = (shared ? a.S3s : a.W3s) + wrow * (d / 32);
                as = a.xs + tok * (d / 32);
            } else if constexpr (ST == ST_FP8) {
                const int64_t srow = ((shared ? 0 : (int64_t)e * a.inter) + f0) / 128 * (d / 128) * 4;
                w1s = (shared ? a.S1s : a.W1s) + srow;
                w3s = (shared ? a.S3s : a.W3s) + srow;
                as = a.xs + tok * (d / 128) * 4;
            }
            const int nun = d / 128, u0 = nun * wave / FEW_NW, u1 = nun * (wave + 1) / FEW_NW;
            f32x4 acc1 = {0.f, 0.f, 0.f, 0.f}, acc3 = {0.f, 0.f, 0.f, 0.f};
            stream_units<ST, true, DU>(acc1, acc3, w1, w1s, w3, w3s, a.x + tok * (d / 128) * TY::abytes + 16 * q, as, u0, u1, q);
            float* red = (float*)buf;
            *(f32x4*)(red + wave * 512 + lane * 4) = acc1;
            *(f32x4*)(red + wave * 512 + 256 + lane * 4) = acc3;
            __syncthreads();
            if (tid < 256) {                           // element tid: token (tid / 4) % 16, feature 4 (tid / 64) + tid % 4
                float gg = 0.f, uu = 0.f;
#pragma unroll
                for (int w = 0; w < FEW_NW; w++) {
                    gg += red[w * 512 + tid];
                    uu += red[w * 512 + 256 + tid];
                }
                const int r = (tid >> 2) & 15, f = f0 + 4 * (tid >> 6) + (tid & 3);
                if constexpr (BF) {
                    round_bf16x2(gg, uu);
                    if (r < n) ((uint16_t*)a.h)[(int64_t)s_slot[g][r] * a.inter_max + f] = f32_to_bf16(silu_mul_fast(gg, uu));
                } else {
                    if (r < n) ((float*)a.h)[(int64_t)s_slot[g][r] * a.inter_max + f] = silu_mul(gg, uu);
                }
            }
            __syncthreads();
            if (tid == 0) __hip_atomic_fetch_add(&a.up_done[g], 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
            continue;
        }

        // ---- 128 output features of one expert: a wavefront takes 16 of them over the whole K
        const int v = item - n_up, g = v / ncol, c = v % ncol;
        const bool shared = g == 0;
        const int e = shared ? 0 : s_exp[g], n = s_n[g], K = shared ? a.inter_s : a.inter;
        const int64_t ldw = (int64_t)(K / 128) * TY::wbytes;
        const int64_t wrow = (shared ? 0 : (int64_t)e * d) + c * FEW_DN + wave * 16 + r16;
        const uint8_t* w2 = (shared ? a.S2 : a.W2) + wrow * ldw + 16 * q;
        const uint8_t* w2s = nullptr;
        if constexpr (ST == ST_MX4) w2s = (shared ? a.S2s : a.W2s) + wrow * (K / 32);
        else if constexpr (ST == ST_FP8)
            w2s = (shared ? a.S2s : a.W2s) + ((shared ? 0 : (int64_t)e * d) + c * FEW_DN + wave * 16) / 128 * (K / 128) * 4;
        const int nun = K / 128;
        WUnit<ST> rw[DD];
#pragma unroll
        for (int j = 0; j < DD; j++) rw[j].load(w2, w2s, min(j, nun - 1));      // these need no h
        if (tid == 0) {
            const int need = shared ? nu_s : nu_r;
            while (__hip_atomic_load(&a.up_done[g], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < need)
                __builtin_amdgcn_s_sleep(1);
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        }
        __syncthreads();
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        const int ar = r16 < n ? r16 : 0;
        for (int u0 = 0; u0 < nun; u0 += KC / 128) {
            const int kc = min(KC, K - u0 * 128);      // elements of this chunk
            if (u0) __syncthreads();                   // the chunk before is used up
            const int vecs = kc / 8;                   // 8 elements a thread; a multiple of 16
            for (int i = tid; i < n * vecs; i += NT) {
                const int r = i / vecs, p = i % vecs;
                const int64_t src = (int64_t)s_slot[g][r] * a.inter_max + u0 * 128 + p * 8;
                if constexpr (ST == ST_F32) {
                    const float4* s = (const float4*)((const float*)a.h + src);
                    *(float4*)(buf + r * HSTR + p * 32) = s[0];
                    *(float4*)(buf + r * HSTR + p * 32 + 16) = s[1];
                } else {
                    const uint4 raw = *(const uint4*)((const uint16_t*)a.h + src);
                    if constexpr (ST == ST_BF16) {
                        *(uint4*)(buf + r * HSTR + p * 16) = raw;
                    } else {
                        float hv[8];
                        bf16x8_to_f32(raw, hv);
                        if constexpr (ST == ST_MX4) {
                            const uint32_t sc = mx_scale_code<false>(quad_max(mx_amax8(hv)));
                            *(uint2*)(buf + r * HSTR + p * 8) = sc == 255u ? make_uint2(0u, 0u) : mx_pack_fp8(hv, sc);
                            if ((p & 3) == 0) hsc[r * (KC / 32) + p / 4] = (uint8_t)sc;
                        } else {
                            float sc;
                            *(uint2*)(buf + r * HSTR + p * 8) = quant8_e4m3(hv, sc);
                            if ((p & 15) == 0) ((float*)hsc)[r * (KC / 128) + p / 16] = sc;
                        }
                    }
                }
            }
            __syncthreads();
            const uint8_t* hb = buf + ar * HSTR + 16 * q;
            const uint8_t* hs = hsc + ar * (ST == ST_MX4 ? KC / 32 : KC / 128 * 4);
            for (int u = 0; u < kc / 128; u += DD) {
#pragma unroll
                for (int j = 0; j < DD; j++) {
                    if (u + j < kc / 128) {
                        AUnit<ST> ra;
                        ra.load(hb, hs, u + j);
                        stream_mma<ST>(acc, rw[j], ra, q);
                        rw[j].load(w2, w2s, min(u0 + u + j + DD, nun - 1));
                    }
                }
            }
        }
        // this lane: features 4 q .. 4 q + 3 of the group's row r16
        if (r16 < n) {
            uint8_t* o = a.y_rows + ((int64_t)s_slot[g][r16] * d + c * FEW_DN + wave * 16 + 4 * q) * AB;
            if constexpr (BF) *(uint2*)o = make_uint2(f32x2_to_bf16x2(acc[0], acc[1]), f32x2_to_bf16x2(acc[2], acc[3]));
            else *(f32x4*)o = acc;
        }
        __syncthreads();
        if (tid == 0)
            s_last = __hip_atomic_fetch_add(&a.col_done[c], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == ng - 1;
        __syncthreads();
        if (s_last) {
            // the experts' outputs for these columns are there: the combine, by ascending expert, then the shared one
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
            constexpr int VE = 16 / AB, VR = FEW_DN / VE;              // elements of a vector, vectors of a row
            for (int i = tid; i < T * VR; i += NT) {
                const int t = i / VR;
                const int64_t col = c * FEW_DN + i % VR * VE;
                float s[VE];
#pragma unroll
                for (int j = 0; j < VE; j++) s[j] = 0.f;
                for (int j = 0; j <= k; j++) {
                    const int sl = j < k ? s_order[t * k + j] : slots + t;
                    const uint4 raw = *(const uint4*)(a.y_rows + ((int64_t)sl * d + col) * AB);
                    const uint32_t wv[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                    for (int m = 0; m < VE; m++) {
                        const float o = BF ? __uint_as_float(m & 1 ? (wv[m / 2] & 0xFFFF0000u) : (wv[m / 2] << 16))
                                           : __uint_as_float(wv[m]);
                        s[m] = j < k ? s[m] + o * s_w[sl] : s[m] + o;
                    }
                }
                uint4 o;
                if constexpr (BF) o = make_uint4(f32x2_to_bf16x2(s[0], s[1]), f32x2_to_bf16x2(s[2], s[3]),
                                                 f32x2_to_bf16x2(s[4], s[5]), f32x2_to_bf16x2(s[6], s[7]));
                else o = make_uint4(__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]), __float_as_uint(s[3]));
                *(uint4*)(a.y + ((int64_t)t * d + col) * AB) = o;
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------------------
struct FewWorkspace {
    float* logits;
    uint8_t *xq, *xs, *h, *y_rows;
    int32_t* counters;
    int n_counters;
    size_t total;
};

static FewWorkspace carve_few(const moe_shape_t& s, void* base)
{
    FewWorkspace w = {};
    const size_t T = (size_t)s.T, d = (size_t)s.d, rows = T * (size_t)s.k + T;
    const size_t act = s.act_dtype == MOE_F32 ? 4 : 2, imax = (size_t)(s.inter > s.inter_shared ? s.inter : s.inter_shared);
    size_t off = 0;
    auto take_bytes = [&](size_t bytes) -> uint8_t* {
        uint8_t* p = base ? (uint8_t*)base + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return p;
    };
    w.n_counters = 1 + FEW_GROUPS + (int)(d / FEW_DN);
    w.counters = (int32_t*)take_bytes(4 * (size_t)w.n_counters);
    w.logits = (float*)take_bytes(4 * T * (size_t)s.E);
    if (s.w_dtype == MOE_FP8_E4M3 || s.w_dtype == MOE_MXFP4) {
        w.xq = take_bytes(T * d);
        w.xs = take_bytes(T * (d / 32));               // E8M0 bytes, or fp32 per 128: the same size
    }
    w.h = take_bytes(rows * imax * act);
    w.y_rows = take_bytes(rows * d * act);
    w.total = off;
    return w;
}

size_t few_workspace_bytes(const moe_shape_t& s) { return carve_few(s, nullptr).total; }

template <int ST, int TM>
static void launch_prepare(const moe_shape_t& s, const void* x, const float* Wg, const float* bias, const FewWorkspace& w,
                           hipStream_t stream)
{
    const bool quant = ST == ST_FP8 || ST == ST_MX4;
    const int nq = quant ? (int)((s.T * s.d / 8 + 255) / 256) : 0;
    few_prepare_kernel<ST, TM><<<(unsigned)(s.E + nq + 1), 256, 0, stream>>>(x, Wg, bias, w.logits, (int)s.T, (int)s.d, (int)s.E,
                                                                             w.xq, w.xs, w.counters, w.n_counters);
}

template <int ST>
static hipError_t launch_few_t(const moe_shape_t& s, const void* x, const float* Wg, const float* bias, FewArgs a,
                               const FewWorkspace& w, hipStream_t stream)
{
    if (s.T == 1) launch_prepare<ST, 1>(s, x, Wg, bias, w, stream);
    else if (s.T == 2) launch_prepare<ST, 2>(s, x, Wg, bias, w, stream);
    else if (s.T <= 4) launch_prepare<ST, 4>(s, x, Wg, bias, w, stream);
    else if (s.T <= 8) launch_prepare<ST, 8>(s, x, Wg, bias, w, stream);
    else launch_prepare<ST, 16>(s, x, Wg, bias, w, stream);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    // two blocks for each of the card's 256 CUs (any number is right: see above)
    few_layer_kernel<ST><<<512, 64 * FEW_NW, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_few(const moe_shape_t& s, const void* x, const float* Wg, const float* bias, const FewWeights& m, void* y,
                      int32_t* idx_out, float* w_out, int32_t* counts_out, void* workspace, hipStream_t stream)
{
    const FewWorkspace w = carve_few(s, workspace);
    const bool quant = s.w_dtype == MOE_FP8_E4M3 || s.w_dtype == MOE_MXFP4;
    FewArgs a = {};
    a.T = (int)s.T;
    a.d = (int)s.d;
    a.E = (int)s.E;
    a.k = (int)s.k;
    a.inter = (int)s.inter;
    a.inter_s = (int)s.inter_shared;
    a.inter_max = (int)(s.inter > s.inter_shared ? s.inter : s.inter_shared);
    a.x = quant ? w.xq : (const uint8_t*)x;
    a.xs = w.xs;
    a.logits = w.logits;
    a.W1 = (const uint8_t*)m.W1;
    a.W3 = (const uint8_t*)m.W3;
    a.W2 = (const uint8_t*)m.W2;
    a.W1s = (const uint8_t*)m.W1s;
    a.W3s = (const uint8_t*)m.W3s;
    a.W2s = (const uint8_t*)m.W2s;
    a.S1 = (const uint8_t*)m.S1;
    a.S3 = (const uint8_t*)m.S3;
    a.S2 = (const uint8_t*)m.S2;
    a.S1s = (const uint8_t*)m.S1s;
    a.S3s = (const uint8_t*)m.S3s;
    a.S2s = (const uint8_t*)m.S2s;
    a.h = w.h;
    a.y_rows = w.y_rows;
    a.y = (uint8_t*)y;
    a.idx_out = idx_out;
    a.w_out_bits = (int32_t*)w_out;
    a.counts_out = counts_out;
    a.ticket = w.counters;
    a.up_done = w.counters + 1;
    a.col_done = w.counters + 1 + FEW_GROUPS;
    if (s.act_dtype == MOE_F32) return launch_few_t<ST_F32>(s, x, Wg, bias, a, w, stream);
    if (s.w_dtype == MOE_FP8_E4M3) return launch_few_t<ST_FP8>(s, x, Wg, bias, a, w, stream);
    if (s.w_dtype == MOE_MXFP4) return launch_few_t<ST_MX4>(s, x, Wg, bias, a, w, stream);
    return launch_few_t<ST_BF16>(s, x, Wg, bias, a, w, stream);
}

}  // namespace moe
