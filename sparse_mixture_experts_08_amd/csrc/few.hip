// few.hip -- the whole layer for at most MOE_FEW_MAX_T tokens in two launches (moe_forward_few).
//
// With so few tokens every weight byte is read once and used for a handful of multiplications: the weights of
// the selected experts bound the layer, and at one token also whatever keeps HBM idle, which is each launch's
// start and drain and each serial step in between.  So:
//   launch 1 (few_prepare_kernel): router logits, one block per expert; the activations' quantisation, where the
//     weight type has one; the counters of launch 2 set to zero.
//   launch 2 (few_layer_kernel): a grid that fills the card once, whose blocks take work items from one counter
//     until none is left.  Every block first selects the experts itself (a top-k over T rows of logits, cheaper
//     than a hand-off between blocks) and keeps x in LDS where it fits.  Items, in this order: the up products of the
//     shared expert and of each selected expert, eight hidden features a wavefront; then their down products, 32
//     output features a wavefront.  A down item waits for its expert's up items, its first weights on their way
//     meanwhile, and the block that completes the last down item of a column range sums the experts' outputs there.
//     No launch boundary lies between the phases.
// Full layer: one token 61 us in MXFP4 (218 MB; 31 us at the 7.1 TB/s of a read alone), 139 us in bf16 (800 MB; 113), four
// tokens in fp8 226 us (1.4 GB; 197), sixteen in MXFP4 156 us (1.1 GB; 160, these few experts partly cached); launch 1
// another 5 to 9 us.  What is lost at one token: the selection (6 us), the wait for the slowest block's h
// and the down jobs' two rounds.
//
// Why every wait ends.  Blocks take item numbers from the counter in ascending order, and an item waits only for
// items of lower numbers.  Take the lowest unfinished item: the block that holds it is running (it took the
// number), and what it held before is finished or under way without a wait, since that has a lower number; what the
// item waits for is finished too; so it completes.  This holds for any number of resident blocks, in any order of
// dispatch, and beside other kernels (a second call of this one among them).  Inside a block, wavefronts wait for
// the number that the first one leaves in LDS; it does so before it waits for anything itself.
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
constexpr int FEW_UP = 8;                              // hidden features a wavefront in an up item
constexpr int FEW_DN = 16 * FEW_NW;                    // output features per down item
constexpr int FEW_PAD = 16;                            // ints between counters: a 64-byte line each
// A group's up jobs are counted in FEW_SUB places: 256 additions to one address at a time take 2 - 5 us in turn (one
// MXFP4 token 66 us with one place, 65 with four or eight; the smallest layer loses to the longer polls with
// more: 30.0 us with eight, 33.7 with 32).
constexpr int FEW_SUB = 4;

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
    int32_t *ticket, *up_done, *col_done;              // counters: [1], [FEW_GROUPS][FEW_SUB], [d / FEW_DN], FEW_PAD apart
};

// ---------------------------------------------------------------------------------------------------
// Launch 1.  Blocks [0, E): the logits of one expert for every token.  Blocks [E, E + nq): quantisation of x.
// The last block clears the counters.
// ---------------------------------------------------------------------------------------------------
constexpr int FEW_NT1 = 1024;                          // threads per block of launch 1

// Eight consecutive elements, raw from the load to their use.
template <typename XT> struct Few8;
template <> struct Few8<uint16_t> {
    uint4 r;
    __device__ __forceinline__ void load(const uint16_t* p) { r = *(const uint4*)p; }
    __device__ __forceinline__ void get(float (&v)[8]) const { bf16x8_to_f32(r, v); }
};
template <> struct Few8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = ((const float4*)p)[0];
        b = ((const float4*)p)[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// Sums of TM values over a wavefront, value t to the lanes whose top log2(TM) bits are t (bit 5 first): each step
// halves the values that a lane keeps and adds the partner's, so TM values take TM - 1 exchanges and then one per
// remaining bit, against 6 TM.
template <int N, int TM> __device__ __forceinline__ void wave_sums_step(double (&v)[TM], int lane, int off)
{
    if constexpr (N >= 1) {
        const bool hi = lane & off;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const double keep = hi ? v[N + i] : v[i], give = hi ? v[i] : v[N + i];
            v[i] = keep + __shfl_xor(give, off, 64);
        }
        wave_sums_step<N / 2, TM>(v, lane, off / 2);
    }
}
template <int TM> __device__ __forceinline__ double wave_sums(double (&v)[TM], int lane)
{
    wave_sums_step<TM / 2, TM>(v, lane, 32);
#pragma unroll
    for (int o = 32 / TM; o >= 1; o >>= 1) v[0] += __shfl_xor(v[0], o, 64);
    return v[0];
}

template <int ST, int TM>
__global__ __launch_bounds__(FEW_NT1) void few_prepare_kernel(const void* __restrict__ xv, const float* __restrict__ Wg,
                                                              const float* __restrict__ bias, float* __restrict__ logits,
                                                              int T, int d, int E, uint8_t* __restrict__ xq,
                                                              uint8_t* __restrict__ xs, int32_t* __restrict__ counters,
                                                              int n_counters)
{
    typedef typename std::conditional<ST == ST_F32, float, uint16_t>::type XT;
    const XT* x = (const XT*)xv;
    const int tid = threadIdx.x, b = blockIdx.x;
    if (b < E) {
        __shared__ double part[FEW_NT1 / 64][TM];
        double acc[TM];
#pragma unroll
        for (int t = 0; t < TM; t++) acc[t] = 0.0;
        const float* wrow = Wg + (size_t)b * d;
        for (int i = tid * 8; i < d; i += 8 * FEW_NT1) {
            constexpr int TC = ST == ST_F32 && TM > 8 ? 8 : TM;        // tokens at a time: their loads first, in flight together
            Few8<float> wr;
            wr.load(wrow + i);
#pragma unroll
            for (int t0 = 0; t0 < TM; t0 += TC) {
                Few8<XT> xr[TC];
#pragma unroll
                for (int t = 0; t < TC; t++) xr[t].load(x + (size_t)min(t0 + t, T - 1) * d + i);
                __builtin_amdgcn_sched_barrier(0);
                float w[8];
                wr.get(w);
#pragma unroll
                for (int t = 0; t < TC; t++) {
                    float v[8];
                    xr[t].get(v);
#pragma unroll
                    for (int e = 0; e < 8; e++) acc[t0 + t] = __builtin_fma((double)v[e], (double)w[e], acc[t0 + t]);
                }
            }
        }
        const int lane = tid & 63;
        const double s = wave_sums<TM>(acc, lane);
        if (lane % (64 / TM) == 0) part[tid >> 6][lane / (64 / TM)] = s;
        __syncthreads();
        if (tid < T) {
            double s = part[0][tid];
#pragma unroll
            for (int w = 1; w < FEW_NT1 / 64; w++) s += part[w][tid];
            if (bias) s += (double)bias[b];
            logits[(size_t)tid * E + b] = (float)s;
        }
        return;
    }
    if (b == (int)gridDim.x - 1) {
        for (int i = tid; i < n_counters; i += FEW_NT1) counters[i] = 0;
        return;
    }
    const int64_t i = (int64_t)(b - E) * FEW_NT1 + tid;                // eight elements each
    if (i >= (int64_t)T * d / 8) return;                               // whole groups of 16 lanes leave together
    float v[8];
    if constexpr (ST == ST_MX4) {
        bf16x8_to_f32(((const uint4*)x)[i], v);
        const uint32_t c = mx_scale_code<false>(quad_max(mx_amax8(v)));
        ((uint2*)xq)[i] = c == 255u ? make_uint2(0u, 0u) : mx_pack_fp8(v, c);
        if ((i & 3) == 0) xs[i >> 2] = (uint8_t)c;
    } else if constexpr (ST == ST_FP8) {
        bf16x8_to_f32(((const uint4*)x)[i], v);
        float sc;
        ((uint2*)xq)[i] = quant8_e4m3(v, sc);
        if ((i & 15) == 0) ((float*)xs)[i >> 4] = sc;
    }
}

// ---------------------------------------------------------------------------------------------------
// Launch 2.
// ---------------------------------------------------------------------------------------------------
// What blocks hand each other (h, expert outputs, counters) is written and read with device-scope accesses, which
// go past the L2 of the writer's XCD to where every XCD sees them.  A producer's wavefronts wait for their stores
// before the barrier behind which one lane raises the counter; a consumer's loads come after the barrier behind
// which that lane has seen it.  (Ordinary stores and a device-scope release instead write back the whole L2 once an
// item.)
typedef unsigned long long u64;
__device__ __forceinline__ void put64(void* p, u64 v) { __hip_atomic_store((u64*)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ u64 get64(const void* p) { return __hip_atomic_load((u64*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint4 get128(const void* p)
{
    const u64 a = get64(p), b = get64((const uint8_t*)p + 8);
    return make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32));
}
// By one lane.  The address is a lane's own as far as the compiler knows: for one that is the wavefront's it adds up
// the lanes first and waits at once for the result, and so for every load of weights before it.
__device__ __forceinline__ int32_t bump(int32_t* counter)
{
    asm volatile("" : "+v"(counter));
    return __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Four consecutive values, rounded to bf16 or as they are.
template <bool BF> __device__ __forceinline__ void put4(uint8_t* p, const float (&v)[4])
{
    if constexpr (BF) {
        put64(p, (u64)f32x2_to_bf16x2(v[0], v[1]) | (u64)f32x2_to_bf16x2(v[2], v[3]) << 32);
    } else {
        put64(p, (u64)__float_as_uint(v[0]) | (u64)__float_as_uint(v[1]) << 32);
        put64(p + 8, (u64)__float_as_uint(v[2]) | (u64)__float_as_uint(v[3]) << 32);
    }
}

// The kernel's argument block (its only argument).
typedef const __attribute__((address_space(4))) FewArgs* KernArgs;

// Bytes of an activation as a linear takes it, and the elements of h that fit LDS at a time.
template <int ST> struct FewAct;
template <> struct FewAct<ST_F32> { static constexpr int bytes = 4; };
template <> struct FewAct<ST_BF16> { static constexpr int bytes = 2; };
template <> struct FewAct<ST_FP8> { static constexpr int bytes = 1; };
template <> struct FewAct<ST_MX4> { static constexpr int bytes = 1; };

// LDS for activations: 16 rows of up to 7168 bytes, each padded so that 16 rows' pieces fall on distinct banks.
// X_LDS: x fits (rows of d elements) and is kept there for the up items.
constexpr int FEW_ROW = 7168, FEW_XBYTES = 16 * (FEW_ROW + STREAM_PAD), FEW_XSCALES = 16 * FEW_ROW / 32;

// First unit of wavefront w's part of nu units, at a multiple of four (a scale load's units).
__device__ __forceinline__ int split_at(int nu, int w) { return min(nu, (nu + 3) / 4 * w / FEW_NW * 4); }

// What a wavefront does next.
struct FewJob {
    int kind, g, at;                                   // group; first hidden feature (up) or column range (down)
};
// FEW_SPLIT_JOB: an up job that the block's wavefronts share, each a part of K.
enum { FEW_NONE = 0, FEW_IDLE = 1, FEW_UP_JOB = 2, FEW_SPLIT_JOB = 3, FEW_DN_JOB = 4 };

template <int ST, bool X_LDS>
__global__ __launch_bounds__(64 * FEW_NW, 2) void few_layer_kernel(FewArgs args)
{
    constexpr bool BF = ST != ST_F32;                  // activations are bf16
    // D weight units in flight a wavefront: eight where x lies in LDS.  Where x travels along from memory, as many as
    // do not spill: four (16 bf16 tokens of a 64-expert layer 737 us, 1178 with eight; 8 fp32 tokens 412 and 532), in
    // MXFP4, whose units hold the most of x, two (16 tokens of d = 7296, 64 experts 408 us, 612 with four).
    constexpr int AB = BF ? 2 : 4, NT = 64 * FEW_NW, LK = StreamType<ST>::K, D = X_LDS ? 8 : ST == ST_MX4 ? 2 : 4;
    constexpr int XB = FewAct<ST>::bytes, HSTR = FEW_ROW + STREAM_PAD;
    constexpr int KC = FEW_ROW / XB / (LK * D) * (LK * D);             // elements of h in LDS at a time: whole rounds
    static_assert(KC > 0, "a round of h fits a row");
    __shared__ __attribute__((aligned(16))) uint8_t act[FEW_XBYTES];   // x; then h
    __shared__ __attribute__((aligned(16))) uint8_t act_s[FEW_XSCALES];        // their scales
    __shared__ __attribute__((aligned(16))) uint8_t tiles[FEW_NW][STREAM_TILE];
    __shared__ int s_idx[FEW_SLOTS];                   // expert of each slot
    __shared__ float s_w[FEW_SLOTS];
    __shared__ uint8_t s_order[FEW_SLOTS];             // a token's slots by ascending expert
    __shared__ uint16_t s_exp[FEW_GROUPS];
    __shared__ uint8_t s_n[FEW_GROUPS];
    __shared__ uint8_t s_slot[FEW_GROUPS][16];         // the slots of a group's rows (group 0, the shared one: tokens)
    __shared__ volatile uint64_t s_ticket[64];         // round + 1 and the item number taken for it, by round % 64
    __shared__ int scan[FEW_NW];                       // selected experts of a wavefront's 128
    __shared__ int s_last;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int T = args.T, k = args.k, E = args.E, d = args.d, slots = T * k;
    const int xstr = d * XB + (X_LDS ? STREAM_PAD : 0); // bytes between rows of x
    const int xsstr = ST == ST_MX4 ? d / 32 : ST == ST_FP8 ? d / 128 * 4 : 0;   // ... of its scales
    int ticket = 0;
    if (tid == 0) ticket = bump(args.ticket);
    Stream<ST, X_LDS, D> st;
    // The arguments are read anew for each job: kept over the loop they would take most scalar registers.
    auto arguments = [&]() -> KernArgs {
        KernArgs p = (KernArgs)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(p));
        return p;
    };
    auto up_rows = [&](const FewJob& job, int& tok, int& slot, int& n) {
        n = __builtin_amdgcn_readfirstlane(s_n[job.g]);
        slot = s_slot[job.g][r16 < n ? r16 : 0];       // lanes past the rows repeat the first
        tok = job.g ? slot / k : slot;
    };
    // The stream goes on with this job's weights.
    auto start = [&](const FewJob& job) {
        const auto& a = *arguments();
        if (job.kind == FEW_UP_JOB || job.kind == FEW_SPLIT_JOB) {     // eight rows of W1 and the same eight of W3
            const int64_t ldw = (int64_t)d * 128 / LK;
            const int e = job.g ? __builtin_amdgcn_readfirstlane(s_exp[job.g]) : 0;
            const int64_t row0 = (int64_t)e * a.inter + job.at;
            const uint8_t* s = nullptr;
            if constexpr (ST == ST_MX4)
                s = (job.g ? (r16 < 8 ? a.W1s : a.W3s) : (r16 < 8 ? a.S1s : a.S3s)) + (row0 + (r16 & 7)) * (d / 32);
            if constexpr (ST == ST_FP8)                // the lane's results are of features 4 q .. 4 q + 3
                s = (job.g ? (q < 2 ? a.W1s : a.W3s) : (q < 2 ? a.S1s : a.S3s)) + row0 / 128 * (d / 128) * 4;
            const int nu = stream_units_of<ST>(d);
            const bool all = job.kind == FEW_UP_JOB;
            st.start(weight_rows<ST>((job.g ? a.W1 : a.S1) + row0 * ldw, (job.g ? a.W3 : a.S3) + row0 * ldw, s, ldw, d, lane),
                     all ? 0 : split_at(nu, wave), all ? nu : split_at(nu, wave + 1));
            if constexpr (!X_LDS) {
                int tok, slot, n;
                up_rows(job, tok, slot, n);
                st.ar = {a.x, a.xs, (uint32_t)tok * xstr + 16 * q, (uint32_t)tok * xsstr, st.wr.half};
            }
        } else if (job.kind == FEW_DN_JOB) {           // 16 rows of W2
            const int K = job.g ? a.inter : a.inter_s;
            const int64_t ldw = (int64_t)K * 128 / LK;
            const int e = job.g ? __builtin_amdgcn_readfirstlane(s_exp[job.g]) : 0;
            const int64_t row0 = (int64_t)e * d + job.at * FEW_DN + wave * 16;
            const uint8_t* s = nullptr;
            if constexpr (ST == ST_MX4) s = (job.g ? a.W2s : a.S2s) + (row0 + r16) * (K / 32);
            if constexpr (ST == ST_FP8) s = (job.g ? a.W2s : a.S2s) + row0 / 128 * (K / 128) * 4;
            const uint8_t* p0 = (job.g ? a.W2 : a.S2) + row0 * ldw;
            st.start(weight_rows<ST>(p0, p0 + 8 * ldw, s, ldw, K, lane), 0, stream_units_of<ST>(K));
            if constexpr (!X_LDS) st.ar = {a.x, a.xs, (uint32_t)(16 * q), 0, 0};       // travels along unused
        } else {
            st.stay();                                 // nothing follows: the last unit again, unused
        }
        if constexpr (!X_LDS) st.ar_step = job.kind == FEW_UP_JOB || job.kind == FEW_SPLIT_JOB;
    };

    // ---- x into LDS, and the selection: every block for itself
    if constexpr (X_LDS) {
        const int vecs = d * XB / 16;                  // 16-byte vectors a row
        for (int i = tid; i < T * vecs; i += NT) {
            const int t = i / vecs;
            *(uint4*)(act + t * xstr + (i - t * vecs) * 16) = ((const uint4*)args.x)[i];
        }
        for (int i = tid; i < T * xsstr / 4; i += NT) ((uint32_t*)act_s)[i] = ((const uint32_t*)args.xs)[i];
    }
    uint32_t* s_tok = (uint32_t*)tiles;                // tokens (bits) of each expert
    uint16_t* s_grp = (uint16_t*)(s_tok + 1024);       // group of each selected expert
    if (tid < 64) s_ticket[tid] = 0;
    s_tok[tid] = s_tok[NT + tid] = 0;
    static_assert(2 * NT == 1024 && NT >= FEW_SLOTS, "two experts a thread, a slot a thread");
    for (int t = wave; t < T; t += FEW_NW) {
        int e;
        float w;
        if (E <= 256) topk_group<64, 4>(args.logits + (size_t)t * E, nullptr, E, k, lane, e, w);
        else topk_group<64, 16>(args.logits + (size_t)t * E, nullptr, E, k, lane, e, w);
        if (lane < k) {
            s_idx[t * k + lane] = e;
            s_w[t * k + lane] = w;
        }
    }
    lds_barrier();
    if (tid < slots) atomicOr(&s_tok[s_idx[tid]], 1u << (tid / k));
    lds_barrier();
    const uint32_t m0 = s_tok[2 * tid], m1 = s_tok[2 * tid + 1];
    // groups 1 ..: the selected experts in ascending order
    const uint64_t b0 = __ballot(m0 != 0), b1 = __ballot(m1 != 0), below = (1ull << lane) - 1;
    if (lane == 0) scan[wave] = __popcll(b0) + __popcll(b1);
    lds_barrier();
    int n_sel = 0, rank = 1 + __popcll(b0 & below) + __popcll(b1 & below);
#pragma unroll
    for (int w = 0; w < FEW_NW; w++) {
        rank += w < wave ? scan[w] : 0;
        n_sel += scan[w];
    }
    n_sel = __builtin_amdgcn_readfirstlane(n_sel);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t m = i ? m1 : m0;
        const int r = i ? rank + (m0 != 0) : rank;
        if (m) {
            s_grp[2 * tid + i] = (uint16_t)r;
            s_exp[r] = (uint16_t)(2 * tid + i);
            s_n[r] = (uint8_t)__popc(m);
        }
    }
    if (tid < 16) s_slot[0][tid] = (uint8_t)min(tid, T - 1);
    if (tid == 0) s_n[0] = (uint8_t)T;
    lds_barrier();
    if (tid < slots) {
        const int t = tid / k, e = s_idx[tid];
        s_slot[s_grp[e]][__popc(s_tok[e] & ((1u << t) - 1u))] = (uint8_t)tid;
        int before = 0;
        for (int j = 0; j < k; j++) before += s_idx[t * k + j] < e;
        s_order[t * k + before] = (uint8_t)tid;
    }
    if (blockIdx.x == 0) {
        if (tid < slots) {
            if (args.idx_out) args.idx_out[tid] = s_idx[tid];
            if (args.w_out_bits) args.w_out_bits[tid] = __float_as_int(s_w[tid]);
        }
        if (args.counts_out)
            for (int e = tid; e < E; e += NT) args.counts_out[e] = __popc(s_tok[e]);
    }
    if (tid == 0) s_ticket[0] = 1ull << 32 | (uint32_t)ticket;
    lds_barrier();

    // ---- jobs.  Numbers of items: n_wide items of FEW_NW wavefronts' up jobs each; then n_split up jobs that a block's
    // wavefronts share; then ng * ncol down items.  Wide items run a block's wavefronts without a joint.  Where the
    // up jobs are not a multiple of the grid's wavefronts, the rest of them as wide items would keep a few blocks
    // busy (at the rate of a few CUs) while most wait for h: a rest of up to one job a block is shared out instead.
    // (One token of the full layer: 2304 jobs on 2048 wavefronts.)
    const int ng = 1 + n_sel, nu_s = args.inter_s / FEW_UP, nu_r = args.inter / FEW_UP, ncol = d / FEW_DN;
    const int n_wup = nu_s + n_sel * nu_r, rest = n_wup % (FEW_NW * (int)gridDim.x);
    const int n_split = rest <= (int)gridDim.x ? rest : 0;
    const int n_wide = (n_wup - n_split + FEW_NW - 1) / FEW_NW, n_up = n_wide + n_split, total = n_up + ng * ncol;
    int round = 0;                                     // of item numbers
    // The block's item of this round: its first lane leaves it in LDS, the other wavefronts find it there.  In the up
    // jobs wavefronts pass from round to round without waiting for each other; the barrier every 32 rounds (below)
    // keeps the fastest from overwriting a number that the slowest has not read.
    auto job_of_round = [&]() -> FewJob {
        uint64_t got;
        while ((int)((got = s_ticket[round % 64]) >> 32) != round + 1) __builtin_amdgcn_s_sleep(1);
        const int item = __builtin_amdgcn_readfirstlane((int)got);
        if (item >= total) return {FEW_NONE, 0, 0};    // every block comes to a number past the end
        if (item >= n_up) return {FEW_DN_JOB, (item - n_up) / ncol, (item - n_up) % ncol};
        const bool wide = item < n_wide;
        const int it = wide ? item * FEW_NW + wave : n_wup - n_split + item - n_wide;
        if (it >= n_wup) return {FEW_IDLE, 0, 0};
        const int kind = wide ? FEW_UP_JOB : FEW_SPLIT_JOB;
        if (it < nu_s) return {kind, 0, it * FEW_UP};
        return {kind, 1 + (it - nu_s) / nu_r, (it - nu_s) % nu_r * FEW_UP};
    };
    auto next_job = [&]() -> FewJob {
        round++;
        if (tid == 0) s_ticket[round % 64] = (uint64_t)(round + 1) << 32 | (uint32_t)ticket;
        return job_of_round();
    };
    // Up items whose h is stored but not yet counted (the counter, or -1): vector memory operations complete in order, so
    // once a later load has been used the stores are done; before a wait for others they are waited for.
    int stored = -1;
    auto count_stored = [&](bool drain) {
        if (stored < 0) return;
        if (drain) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (lane == 0) bump(&arguments()->up_done[stored * FEW_PAD]);
        stored = -1;
    };
    // The down item whose column count is on its way (column range, or -1).
    int counted = -1, count = 0;
    // Sums the experts' outputs of that item's columns if it was their last: by ascending expert, then the shared one.
    // Every wavefront comes here; behind a barrier.
    auto combine_if_last = [&] {
        if (counted < 0) return;
        if (s_last) {
            const auto& a = *arguments();
            constexpr int VE = 16 / AB;                // elements of a vector
            constexpr int VR = FEW_DN / VE;            // vectors of a row
            for (int i = tid; i < T * VR; i += NT) {
                const int t = i / VR;
                const int64_t col = counted * FEW_DN + i % VR * VE;
                float sum[VE];
#pragma unroll
                for (int j = 0; j < VE; j++) sum[j] = 0.f;
                for (int j = 0; j <= k; j++) {
                    const int sl = j < k ? s_order[t * k + j] : slots + t;
                    const uint4 raw = get128(a.y_rows + ((int64_t)sl * d + col) * AB);
                    const uint32_t wv[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                    for (int m = 0; m < VE; m++) {
                        const float o = BF ? __uint_as_float(m & 1 ? (wv[m / 2] & 0xFFFF0000u) : (wv[m / 2] << 16))
                                           : __uint_as_float(wv[m]);
                        sum[m] = j < k ? sum[m] + o * s_w[sl] : sum[m] + o;
                    }
                }
                uint4 o;
                if constexpr (BF) o = make_uint4(f32x2_to_bf16x2(sum[0], sum[1]), f32x2_to_bf16x2(sum[2], sum[3]),
                                                 f32x2_to_bf16x2(sum[4], sum[5]), f32x2_to_bf16x2(sum[6], sum[7]));
                else o = make_uint4(__float_as_uint(sum[0]), __float_as_uint(sum[1]), __float_as_uint(sum[2]), __float_as_uint(sum[3]));
                *(uint4*)(a.y + ((int64_t)t * d + col) * AB) = o;
            }
        }
        counted = -1;
    };

    FewJob job = job_of_round();
    bool filled = false;                               // the job's first units are on their way
    while (job.kind != FEW_NONE) {
        if (round % 32 == 31) __syncthreads();
        if (!filled && job.kind != FEW_IDLE) {
            start(job);
            st.fill(lane);
        }
        if (tid == 0) ticket = bump(arguments()->ticket);
        if (job.kind == FEW_IDLE) {
            job = next_job();
            filled = false;
            continue;
        }
        const bool dn = job.kind == FEW_DN_JOB, split = job.kind == FEW_SPLIT_JOB;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        FewJob then;
        int tok = 0, slot = 0, n, K = d;
        if (dn) {
            const auto& a = *arguments();
            n = __builtin_amdgcn_readfirstlane(s_n[job.g]);
            K = job.g ? a.inter : a.inter_s;
            count_stored(true);                        // before the wait: it may be for these
            if (wave == 0) {
                const int need = job.g ? nu_r : nu_s;
                for (;;) {
                    const int32_t* c = &a.up_done[(job.g * FEW_SUB + lane % FEW_SUB) * FEW_PAD];
                    int sum = __hip_atomic_load(c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                    for (int o = 1; o < FEW_SUB; o *= 2) sum += __shfl_xor(sum, o, 64);
                    if (__builtin_amdgcn_readfirstlane(sum) >= need) break;
                    __builtin_amdgcn_s_sleep(64);      // polls from every block delay the weights of those that work
                }
                if (lane == 0) s_last = count == ng - 1;
            }
            __syncthreads();                           // also: every wavefront is past the up jobs, x is not needed any more
            combine_if_last();
        } else {
            up_rows(job, tok, slot, n);
        }
        // One loop for both kinds of job, so that its code is fetched once: a down job's h comes in chunks of KC elements,
        // an up job's x is there.  Before the last round the stream is told what follows.
        for (int k0 = 0, more = 1; more; k0 += KC) {
            ARows al = {act, act_s, (uint32_t)tok * xstr + 16 * q, (uint32_t)tok * xsstr, st.wr.half};
            const int nu = stream_units_of<ST>(K);
            int u0 = split ? split_at(nu, wave) : 0, u1 = split ? split_at(nu, wave + 1) : nu, ua = 0;
            if (dn) {
                // elements [k0, k0 + kc) of the group's rows of h into LDS, as the linear takes them
                const auto& a = *arguments();
                const int kc = min(KC, K - k0), vecs = kc / 8;         // 8 elements a thread; a multiple of 16
                if (k0) __syncthreads();               // the chunk before is used up
                for (int i = tid; i < n * vecs; i += NT) {
                    const int r = i / vecs, p = i - r * vecs, sl = s_slot[job.g][r];
                    const uint8_t* src = a.h + ((int64_t)(job.g ? sl : slots + sl) * a.inter_max + k0 + p * 8) * AB;
                    uint8_t* dst = act + r * HSTR;
                    if constexpr (ST == ST_F32) {
                        *(uint4*)(dst + p * 32) = get128(src);
                        *(uint4*)(dst + p * 32 + 16) = get128(src + 16);
                    } else {
                        const uint4 raw = get128(src);
                        if constexpr (ST == ST_BF16) {
                            *(uint4*)(dst + p * 16) = raw;
                        } else {
                            float hv[8];
                            bf16x8_to_f32(raw, hv);
                            if constexpr (ST == ST_MX4) {
                                const uint32_t sc = mx_scale_code<false>(quad_max(mx_amax8(hv)));
                                *(uint2*)(dst + p * 8) = sc == 255u ? make_uint2(0u, 0u) : mx_pack_fp8(hv, sc);
                                if ((p & 3) == 0) act_s[r * (KC / 32) + p / 4] = (uint8_t)sc;
                            } else {
                                float sc;
                                *(uint2*)(dst + p * 8) = quant8_e4m3(hv, sc);
                                if ((p & 15) == 0) ((float*)act_s)[r * (KC / 128) + p / 16] = sc;
                            }
                        }
                    }
                }
                __syncthreads();
                const int ar = r16 < n ? r16 : 0;
                al = {act, act_s, (uint32_t)(ar * HSTR + 16 * q), (uint32_t)(ar * (ST == ST_MX4 ? KC / 32 : KC / 128 * 4)),
                      ST == ST_MX4 && kc % 256 ? kc / 256 : -1};
                u0 = ua = k0 / LK;
                u1 = u0 + stream_units_of<ST>(kc);
                more = k0 + kc < K;
            } else {
                more = 0;
            }
            for (int u = u0;; u += D) {
                const bool last = u + D >= u1;
                if (last && !more) {
                    then = next_job();
                    start(then);
                }
                if constexpr (X_LDS) {
                    st.template round<true>(acc, al, u, u1, ua, tiles[wave], lane);
                } else {
                    if (dn) st.template round<true, true>(acc, al, u, u1, ua, tiles[wave], lane);
                    else st.template round<true>(acc, al, u, u1, ua, tiles[wave], lane);
                }
                if (last) break;
            }
            if (!dn) count_stored(u1 - u0 <= D);
        }
        filled = then.kind != FEW_IDLE;
        const auto& a = *arguments();
        if (dn) {
            // this lane: features 4 q .. 4 q + 3 of the group's row r16
            if (r16 < n) {
                const int sl = s_slot[job.g][r16];
                const float o[4] = {acc[0], acc[1], acc[2], acc[3]};
                put4<BF>(a.y_rows + ((int64_t)(job.g ? sl : slots + sl) * d + job.at * FEW_DN + wave * 16 + 4 * q) * AB, o);
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (tid == 0) count = bump(&a.col_done[job.at * FEW_PAD]);
            counted = job.at;
        } else {
            bool mine = true;                          // this wavefront has the sums
            if (split) {                               // the parts, joined in their order by the first wavefront
                *(f32x4*)(tiles[wave] + lane * 16) = acc;
                lds_barrier();
                if (wave == 0) {
#pragma unroll
                    for (int w = 1; w < FEW_NW; w++) acc += *(const f32x4*)(tiles[w] + lane * 16);
                }
                lds_barrier();
                mine = wave == 0;
            }
            if (mine) {
                // lanes of q = 0, 1 hold g and those of q = 2, 3 u of features 4 (q % 2) + r
                float hv[4];
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    float gg = acc[r], uu = __shfl_xor(acc[r], 32, 64);
                    if constexpr (BF) {
                        round_bf16x2(gg, uu);
                        hv[r] = silu_mul_fast(gg, uu);
                    } else {
                        hv[r] = silu_mul(gg, uu);
                    }
                }
                if (q < 2 && r16 < n) put4<BF>(a.h + ((int64_t)(job.g ? slot : slots + slot) * a.inter_max + job.at + 4 * q) * AB, hv);
                stored = job.g * FEW_SUB + job.at / FEW_UP % FEW_SUB;
            }
        }
        job = then;
    }
    count_stored(true);
    if (counted >= 0) {
        if (tid == 0) s_last = count == ng - 1;
        __syncthreads();
        combine_if_last();
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
    w.n_counters = (1 + FEW_GROUPS * FEW_SUB + (int)(d / FEW_DN)) * FEW_PAD;
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
    const int nq = quant ? (int)((s.T * s.d / 8 + FEW_NT1 - 1) / FEW_NT1) : 0;
    few_prepare_kernel<ST, TM><<<(unsigned)(s.E + nq + 1), FEW_NT1, 0, stream>>>(x, Wg, bias, w.logits, (int)s.T, (int)s.d, (int)s.E,
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
    // a block for each of the card's 256 CUs (any number is right: see above)
    const int64_t row = s.d * FewAct<ST>::bytes + STREAM_PAD;  // of x in LDS
    if (s.T * row <= FEW_XBYTES && s.T * s.d / 32 <= FEW_XSCALES) few_layer_kernel<ST, true><<<256, 64 * FEW_NW, 0, stream>>>(a);
    else few_layer_kernel<ST, false><<<256, 64 * FEW_NW, 0, stream>>>(a);
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
    a.up_done = w.counters + FEW_PAD;
    a.col_done = w.counters + (1 + FEW_GROUPS * FEW_SUB) * FEW_PAD;
    if (s.act_dtype == MOE_F32) return launch_few_t<ST_F32>(s, x, Wg, bias, a, w, stream);
    if (s.w_dtype == MOE_FP8_E4M3) return launch_few_t<ST_FP8>(s, x, Wg, bias, a, w, stream);
    if (s.w_dtype == MOE_MXFP4) return launch_few_t<ST_MX4>(s, x, Wg, bias, a, w, stream);
    return launch_few_t<ST_BF16>(s, x, Wg, bias, a, w, stream);
}

}  // namespace moe
