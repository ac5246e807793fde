// mx_gemm.hip -- grouped expert GEMMs with MXFP4 weights: the up GEMM (W1, W3, SiLU * mul) and the down GEMM (W2)
// of the layer, over the same tile list as the other types' (see gemm.hip).
//
// Activations enter a linear as MXFP8 (E4M3 codes, one E8M0 scale per 32): x is quantised before the up GEMM, h
// (after its rounding to bf16) in the up GEMM's epilogue.  The product is v_mfma_scale_f32_16x16x128_f8f6f4 with
// E2M1 weights as the first operand and E4M3 activations as the second; the instruction applies both scales
// and adds to the fp32 accumulator, so nothing is rescaled on the vector ALU.  Operand and scale layouts of the
// instruction: see stream.h.
#include "gemm.h"
#include "stream.h"

namespace moe {

// Scale pointers of GemmArgs hold E8M0 bytes here; ldas, ldos and nkb_s count bytes.
static __device__ __forceinline__ const uint8_t* bytes(const float* p) { return (const uint8_t*)p; }

// The group's matrices for one block's output features [n0, ..): rows of K / 2 bytes and K / 32 scale bytes.
struct MxGroup {
    const uint8_t *W1, *W3, *W1s, *W3s;
    int64_t ldb;                                       // bytes between weight rows
    int nkb;                                           // bytes between scale rows
};
template <bool UP> __device__ __forceinline__ MxGroup mx_group(const GemmArgs& g, int grp, bool shared, int N, int K)
{
    MxGroup m;
    const int64_t lgrp = grp - g.e_base;
    m.ldb = (shared ? g.ld_s : (int64_t)K) / 2;
    m.nkb = shared ? g.nkb_s : K / 32;
    m.W1 = shared ? g.S1 : g.B1 + lgrp * N * m.ldb;
    m.W1s = shared ? bytes(g.S1s) : bytes(g.B1s) + lgrp * N * m.nkb;
    m.W3 = UP ? (shared ? g.S3 : g.B3 + lgrp * N * m.ldb) : m.W1;
    m.W3s = UP ? (shared ? bytes(g.S3s) : bytes(g.B3s) + lgrp * N * m.nkb) : m.W1s;
    return m;
}

// ---------------------------------------------------------------------------------------------------
// 16-row tiles (decode): weight bytes bound it.  A block is one tile x 256 output features for the down GEMM, 128
// for the up GEMM; each of its 16 wavefronts streams 16 weight rows (up: eight of W1 and the same eight of W3) over
// the whole K, the tile's activation rows in LDS (up to XK elements of K at a time).
// 64 tokens of the full layer (222 experts, 5.2 GB): up 565 us, down 295 us, 6.1 TB/s.  With loads in operand order (16
// rows x 64 bytes an instruction) and the activations from memory it was 1228 and 611 us.
// ---------------------------------------------------------------------------------------------------
template <bool UP>
__global__ __launch_bounds__(1024, 4) void mx_gemm_stream_kernel(GemmArgs g)
{
    constexpr int NW = 16, NT = 64 * NW, FW = UP ? 8 : 16, BN = NW * FW, D = 4;
    constexpr int XK = UP ? 7168 : 4096, XSTR = XK + STREAM_PAD;       // whole rounds of D units
    static_assert(XK % (D * 256) == 0, "a chunk of K is whole rounds");
    __shared__ __attribute__((aligned(16))) uint8_t xb[16 * XSTR];
    __shared__ __attribute__((aligned(16))) uint8_t xs[16 * (XK / 32)];
    __shared__ __attribute__((aligned(16))) uint8_t tiles[NW][STREAM_TILE];
    static_assert(16 * (BN + 4) * 4 <= NW * STREAM_TILE, "the output tile replaces the weight tiles");

    int tile, nb;
    if (!block_work(g, tile, nb)) return;
    const int4 td = g.tiles[tile];
    const int grp = td.x, row0 = td.y, rows = td.z;
    const bool shared = grp == g.E;
    const int N = shared ? g.N_s : g.N_r, K = shared ? g.K_s : g.K_r;
    const int n0 = nb * BN;
    if (n0 >= N) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const MxGroup m = mx_group<UP>(g, grp, shared, N, K);

    // N is a multiple of 128: the down GEMM's last block may be half there (its other wavefronts repeat the first)
    const bool mine = n0 + wave * FW < N;
    const int64_t w0 = mine ? n0 + wave * FW : n0;     // the wavefront's first feature
    const uint8_t* p0 = m.W1 + w0 * m.ldb;
    const uint8_t* s = UP ? (r16 < 8 ? m.W1s : m.W3s) + (w0 + (r16 & 7)) * m.nkb : m.W1s + (w0 + r16) * m.nkb;
    const WRows wr = weight_rows<ST_MX4>(p0, UP ? m.W3 + w0 * m.ldb : p0 + 8 * m.ldb, s, m.ldb, K, lane);
    const int nu = stream_units_of<ST_MX4>(K);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    Stream<ST_MX4, true, D> st;
    for (int k0 = 0; k0 < K; k0 += XK) {
        const int kc = min(XK, K - k0), vecs = kc / 16;
        if (k0) __syncthreads();                       // the chunk before is used up
        for (int i = tid; i < rows * vecs; i += NT) {
            const int r = i / vecs, p = i - r * vecs;
            const int64_t arow = UP ? g.row_token[row0 + r] : row0 + r;
            *(uint4*)(xb + r * XSTR + p * 16) = *(const uint4*)(g.A + arow * g.lda + k0 + p * 16);
        }
        for (int i = tid; i < rows * (kc / 128); i += NT) {
            const int r = i / (kc / 128), p = i - r * (kc / 128);
            const int64_t arow = UP ? g.row_token[row0 + r] : row0 + r;
            *(uint32_t*)(xs + r * (XK / 32) + p * 4) = *(const uint32_t*)(bytes(g.As) + arow * g.ldas + k0 / 32 + p * 4);
        }
        if (k0 == 0) {                                 // behind the activations' loads, so that these do not wait for it
            st.start(wr, 0, nu);
            st.fill(lane);
        }
        lds_barrier();
        const int ar = r16 < rows ? r16 : 0;           // lanes past the tile's rows repeat its first row (never stored)
        const ARows a = {xb, xs, (uint32_t)(ar * XSTR + 16 * q), (uint32_t)(ar * (XK / 32)), kc % 256 ? kc / 256 : -1};
        const int u0 = k0 / 256, u1 = u0 + stream_units_of<ST_MX4>(kc);
        int u = u0;
        for (; u < u1 && u + D < nu; u += D) st.template round<true>(acc, a, u, u1, u0, tiles[wave], lane);
        if (u < u1) st.template round<false>(acc, a, u, u1, u0, tiles[wave], lane);
    }
    __syncthreads();

    // [token][feature] through LDS, then whole rows: h quantised per 32 features, or y rounded to bf16
    float* hs = (float*)tiles;                         // [16][BN + 4]
    if constexpr (UP) {
        // lanes of q = 0, 1 hold g and those of q = 2, 3 u of features 4 (q % 2) + r
#pragma unroll
        for (int r = 0; r < 4; r++) {
            float gg = acc[r], uu = __shfl_xor(acc[r], 32, 64);
            round_bf16x2(gg, uu);
            acc[r] = round_bf16(silu_mul_fast(gg, uu));
        }
        if (q < 2) *(f32x4*)(hs + r16 * (BN + 4) + wave * 8 + 4 * q) = acc;
    } else {
        *(f32x4*)(hs + r16 * (BN + 4) + wave * 16 + 4 * q) = acc;
    }
    __syncthreads();
    constexpr int TR = BN / 8;                         // threads a row, 8 features each
    const int row = tid / TR, sub = tid % TR;
    if (row < rows && n0 + sub * 8 < N) {              // rows <= 16
        float v[8];
        *(f32x4*)&v[0] = *(const f32x4*)(hs + row * (BN + 4) + sub * 8);
        *(f32x4*)&v[4] = *(const f32x4*)(hs + row * (BN + 4) + sub * 8 + 4);
        const int64_t orow = (int64_t)row0 + row;
        if constexpr (UP) {
            const uint32_t c = mx_scale_code<false>(quad_max(mx_amax8(v)));
            *(uint2*)(g.out + orow * g.ldo + n0 + sub * 8) = c == 255u ? make_uint2(0u, 0u) : mx_pack_fp8(v, c);
            if ((sub & 3) == 0) ((uint8_t*)g.outs)[orow * g.ldos + (n0 + sub * 8) / 32] = (uint8_t)c;
        } else {
            *(uint4*)(g.out + (orow * g.ldo + n0 + sub * 8) * 2) =
                make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                           f32x2_to_bf16x2(v[6], v[7]));
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// 256-row tiles.  Operands and scales are staged through LDS by direct-to-LDS loads; a K stage is 128 elements: 128
// bytes of every activation row, 64 of every weight row (both swizzled by row: see gemm.h).  Activations are
// staged 64 rows at a time, as many as the tile has, and what a stage leaves free becomes further stages of the
// ring (three with 256 rows, six with 64).
//
// Scales are staged for four stages at once (SC16: 16 bytes of each row by one load; otherwise, where scale rows are
// not whole 16-byte words, four planes of 4 bytes): one load of 4 bytes per row and stage fetched a
// line per row each time and took as long as all the rest (the 4096-token layer 3.07 -> 2.44 ms without it).  A lane
// turns them into one register per 16-row block that holds the stages' bytes; the instruction picks one.
//
// Eight wavefronts, 4 (rows) x 2 (features), two to a SIMD, which take turns: while one reads the fragments of a
// stage into registers, the other one multiplies.  Barriers separate the turns, wavefronts 4-7 being one turn
// behind (in step with each other, all reading, then all multiplying: up GEMM of 16384 tokens 4.93 against 3.80 ms).
// Row blocks (16 rows) are dealt to the row groups in turn, so a short tile still spreads over all.
//
// Full layer, 4096 tokens (144 rows a tile): up 1232 us, down 681 us; 16384 skewed tokens: 3707 and 1958 us, 2.3 PFLOP/s.
// A stage's loads (48 KB a CU for 256 rows, mostly from L2) take about as long as its products; the
// 4096-token up GEMM takes 944 us without loads in the loop, and about 1160 us with loads alone.
// ---------------------------------------------------------------------------------------------------
constexpr int MX_BM = 256, MX_RING = 3 * (MX_BM * 128 + 256 * 64);

// Byte offset of 16-byte chunk c of LDS row r, of 128 and of 64 bytes.  A 16-byte read takes 16 lanes a clock: lanes
// 0-3, 12-15 and 20-27, then 4-11, 16-19 and 28-31, and so on.  With lane = row + 16 chunk that is half of the 16 rows
// at one chunk and the other half at the next, which these orders place on all 64 banks.  (gemm.h's order is made for
// 32 rows at one chunk; with it 45 % of the reads' clocks were conflicts and the down GEMM of
// 16384 tokens took 2.49 instead of 1.99 ms.)
__device__ __forceinline__ int mx_swz128(int r, int c) { return r * 128 + ((c ^ (r >> 1 & 7)) << 4); }
__device__ __forceinline__ int mx_swz64(int r, int c) { return r * 64 + ((c ^ (r >> 2 & 3)) << 4); }

template <bool UP, int BN, bool SC16>
__global__ __launch_bounds__(512, 2) void mx_gemm_kernel(GemmArgs g)
{
    constexpr int BM = MX_BM;
    constexpr int NB = UP ? 2 * BN : BN;               // weight rows per stage
    constexpr int WM = BM / 64, WB = NB / 32;          // 16-row blocks per wavefront: activations, weights
    constexpr int WN = BN / 32;                        // ... of one matrix
    constexpr int PB = NB / 128;                       // 1-KB loads of weights per wavefront and stage
    static_assert(!UP || BN == 128, "a wavefront has 64 features of h");
    static_assert(NB == 128 || NB == 256, "whole loads, and scales of 256 + NB rows");
    constexpr int OSTR = (UP ? BN : BN * 2) + 16;      // epilogue: padded LDS row of the output tile
    static_assert(BM * OSTR <= MX_RING, "the output tile replaces the stages");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[MX_RING];
    __shared__ __attribute__((aligned(1024))) uint8_t scl[512 * 16];   // SC16: [row][stage % 4], else [stage % 4][row]
    __shared__ int s_tok[BM];

    int tile, nb;
    if (!block_work(g, tile, nb)) return;
    const int4 td = g.tiles[tile];
    const int grp = td.x, row0 = td.y, rows = td.z;
    const bool shared = grp == g.E;
    const int N = shared ? g.N_s : g.N_r, K = shared ? g.K_s : g.K_r;
    const int n0 = nb * BN;
    if (n0 >= N) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // wavefronts w and w + 4 share a SIMD: row groups 0 and 3, or 1 and 2
    const int late = wave >> 2, mg = late ? 3 - (wave & 1) : wave & 1, ng = (wave >> 1) & 1;
    const int r16 = lane & 15, q = lane >> 4;
    const MxGroup m = mx_group<UP>(g, grp, shared, N, K);

    // rows past the tile's end repeat its first row (valid memory; computed or skipped, never stored)
    if (tid < BM) s_tok[tid] = UP ? g.row_token[row0 + (tid < rows ? tid : 0)] : row0 + (tid < rows ? tid : 0);
    __syncthreads();

    // Sources, fixed over the K walk (32-bit offsets: the host keeps every operand under 4 GB).  Lane l of a load
    // writes 16-byte chunk l % 8 of row l / 8 (activations) or l % 4 of row l / 4 (weights) and so reads the
    // logical chunk that the swizzle keeps there.
    uint32_t offA[WM], offB[PB];
#pragma unroll
    for (int p = 0; p < WM; p++) {
        const int row = (p * 8 + wave) * 8 + (lane >> 3);
        offA[p] = (uint32_t)s_tok[row] * (uint32_t)g.lda + (mx_swz128(row, lane & 7) - row * 128);
    }
#pragma unroll
    for (int p = 0; p < PB; p++) {
        const int row = (p * 8 + wave) * 16 + (lane >> 2);             // UP: rows BN .. are W3's
        offB[p] = (uint32_t)(n0 + (UP ? row % BN : row)) * (uint32_t)m.ldb + (mx_swz64(row, lane & 3) - row * 64);
    }
    // scales: wavefronts 0-3 the activation rows', 4-7 the weight rows' (NB = 128: 6 and 7 repeat 4 and 5)
    uint32_t offS;
    const uint8_t* baseS;
    if (wave < 4) {
        offS = (uint32_t)s_tok[wave * 64 + lane] * (uint32_t)g.ldas;
        baseS = bytes(g.As);
    } else {
        const int row = ((wave - 4) * 64 + lane) % NB;
        offS = (uint32_t)(n0 + row % BN) * (uint32_t)m.nkb;
        baseS = UP && ((wave - 4) * 64) % NB >= BN ? m.W3s : m.W1s;    // BN is a multiple of 64: wave-uniform
    }
    const int nstages = K / 128;
    const uint32_t ring0 = lds_addr(ring), scl0 = lds_addr(scl);
    auto issue_scales = [&](int c) {                   // of stages 4 c .. 4 c + 3; past the end: the last again
        if constexpr (SC16) dma16(baseS + (int64_t)min(c, (nstages - 1) / 4) * 16, offS, scl0 + wave * 1024);
        else
#pragma unroll
            for (int j = 0; j < 4; j++)
                dma4(baseS + (int64_t)min(4 * c + j, nstages - 1) * 4, offS, scl0 + j * 2048 + wave * 256);
    };

    // Fragments in a stage: the row blocks of a wavefront are multiples of 16 rows apart, and the orders repeat
    // every 16 rows.
    const int a_lo = mx_swz128(16 * mg + r16, q), a_hi = mx_swz128(16 * mg + r16, 4 + q);
    const int w_at = mx_swz64(ng * (BN / 2) + r16, q);
    constexpr int SROW = SC16 ? 16 : 4;                // bytes between rows' scales
    const int a_sc = (16 * mg + r16) * SROW, w_sc = (BM + ng * (BN / 2) + r16) * SROW;

    auto k_walk = [&](auto nr_tag) {
        constexpr int NR = decltype(nr_tag)::value;    // 64-row steps of the tile
        if constexpr (NR > 0) {
            constexpr int STAGE = NR * 8192 + NB * 64, FIT = MX_RING / STAGE, NSTG = FIT < 6 ? FIT : 6;
            constexpr int NL = NR + PB;                // loads per wavefront and stage
            static_assert(NSTG >= 3 && (NSTG - 2) * NL < 64, "two stages ahead; vmcnt range");
            f32x4 acc[NR][WB];                                 // UP: features of W1, then of W3
#pragma unroll
            for (int i = 0; i < NR; i++)
#pragma unroll
                for (int j = 0; j < WB; j++) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
            const bool last = 16 * (4 * (NR - 1) + mg) < rows;         // the last step's block has rows (wave-uniform)
            auto issue = [&](int buf, int s) {
                const uint32_t dst = ring0 + buf * STAGE + wave * 1024;
                const int ks = min(s, nstages - 1);    // past the end: the last stage again (never read)
#pragma unroll
                for (int p = 0; p < NR; p++) dma16(g.A + (int64_t)ks * 128, offA[p], dst + p * 8192);
#pragma unroll
                for (int p = 0; p < PB; p++)
                    dma16((UP && p * 128 >= BN ? m.W3 : m.W1) + (int64_t)ks * 64, offB[p], dst + NR * 8192 + p * 8192);
            };
            uint32_t as[NR], ws[WB];
            // One stage.  Its fragments are read in the first turn; the loads issued there go to the buffer of the
            // stage before, which every wavefront has read (the other half in the turn before this one).  Before
            // wavefronts 0-3 begin on the next stage it has landed for all: what may still be on its way then is
            // the NSTG - 2 stages behind it.  That moment is the end of their own second turn and of the others'
            // first.  Scales are read at the first of four stages and loaded again at the second, by when
            // both halves have read them; at the fourth, when they must be there, two stages' loads are younger.
            auto stage = [&](auto j_tag, int s, int& buf) {
                constexpr int J = decltype(j_tag)::value;
                constexpr int BEHIND = (J == 3 && NSTG > 4 ? 2 : NSTG - 2) * NL;
                const uint8_t* sa = ring + buf * STAGE;
                const uint8_t* sb = sa + NR * 8192;
                if constexpr (J == 0) {
                    const uint32_t sel = 0x0c0c0400u + 0x0101u * (uint32_t)q;  // byte q of two words
                    auto gather = [&](const uint8_t* p) {
                        uint32_t w[4];
                        if constexpr (SC16) {
                            const uint4 v = *(const uint4*)p;
                            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; e++) w[e] = *(const uint32_t*)(p + e * 2048);
                        }
                        return __builtin_amdgcn_perm(w[1], w[0], sel) | __builtin_amdgcn_perm(w[3], w[2], sel) << 16;
                    };
#pragma unroll
                    for (int i = 0; i < NR; i++) as[i] = gather(scl + a_sc + 64 * i * SROW);
#pragma unroll
                    for (int j = 0; j < WB; j++) ws[j] = gather(scl + w_sc + ((j / WN) * BN + 16 * (j % WN)) * SROW);
                }
                i32x4 b[WB];
                i32x8 a[NR];
#pragma unroll
                for (int j = 0; j < WB; j++)
                    b[j] = *(const i32x4*)(sb + w_at + ((j / WN) * BN + 16 * (j % WN)) * 64);
#pragma unroll
                for (int i = 0; i < NR; i++) {
                    const i32x4 lo = *(const i32x4*)(sa + a_lo + 64 * i * 128), hi = *(const i32x4*)(sa + a_hi + 64 * i * 128);
                    a[i] = (i32x8){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                }
                issue(buf == 0 ? NSTG - 1 : buf - 1, s + NSTG - 1);
                if constexpr (J == 1) issue_scales(s / 4 + 1);
                if (late) wait_vmcnt<BEHIND>();
                lds_barrier();
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int i = 0; i < NR; i++) {
                    if (i < NR - 1 || last) {
#pragma unroll
                        for (int j = 0; j < WB; j++) {
                            const i32x8 w = {b[j].x, b[j].y, b[j].z, b[j].w, 0, 0, 0, 0};
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a[i], acc[i][j], 4, 0, J, (int)ws[j], J, (int)as[i]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < NR; i++)
#pragma unroll
                    for (int j = 0; j < WB; j++) asm volatile("" : "+v"(acc[i][j]));   // the products stay in this turn
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                if (!late) wait_vmcnt<BEHIND>();
                lds_barrier();
                buf = buf + 1 == NSTG ? 0 : buf + 1;
            };
            issue_scales(0);
#pragma unroll
            for (int t = 0; t < NSTG - 1; t++) issue(t, t);
            wait_vmcnt<(NSTG - 2) * NL>();
            lds_barrier();
            if (late) lds_barrier();                   // half a stage behind
            int buf = 0;
            for (int s = 0; s < nstages; s += 4) {
                stage(IntC<0>{}, s, buf);
                if (s + 1 < nstages) stage(IntC<1>{}, s + 1, buf);
                if (s + 2 < nstages) stage(IntC<2>{}, s + 2, buf);
                if (s + 3 < nstages) stage(IntC<3>{}, s + 3, buf);
            }
            if (!late) lds_barrier();
            wait_vmcnt<0>();                           // no load may still target this block's LDS
            lds_barrier();
            // the output tile into LDS, of the steps that the tile has
            if constexpr (UP) {
                // h of a token's 32 features lies on the four lanes r16 + 16 q, eight values each
#pragma unroll
                for (int i = 0; i < NR; i++) {
                    const int row = 16 * (4 * i + mg) + r16;
#pragma unroll
                    for (int p = 0; p < WN / 2; p++) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            float gg = acc[i][2 * p + e / 4][e % 4], uu = acc[i][WN + 2 * p + e / 4][e % 4];
                            round_bf16x2(gg, uu);
                            v[e] = round_bf16(silu_mul_fast(gg, uu));
                        }
                        uint32_t am = mx_amax8(v);
                        am = max(am, (uint32_t)__shfl_xor((int)am, 16, 64));
                        am = max(am, (uint32_t)__shfl_xor((int)am, 32, 64));
                        const uint32_t c = mx_scale_code<false>(am);
                        const uint2 pk = c == 255u ? make_uint2(0u, 0u) : mx_pack_fp8(v, c);
                        const int f = ng * 64 + p * 32;
                        *(uint32_t*)(ring + row * OSTR + f + 4 * q) = pk.x;
                        *(uint32_t*)(ring + row * OSTR + f + 16 + 4 * q) = pk.y;
                        if (q == 0 && row < rows) ((uint8_t*)g.outs)[((int64_t)row0 + row) * g.ldos + (n0 + f) / 32] = (uint8_t)c;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < NR; i++) {
#pragma unroll
                    for (int j = 0; j < WB; j++) {
                        const uint32_t lo = f32x2_to_bf16x2(acc[i][j][0], acc[i][j][1]);
                        const uint32_t hi = f32x2_to_bf16x2(acc[i][j][2], acc[i][j][3]);
                        *(uint2*)(ring + (16 * (4 * i + mg) + r16) * OSTR + (ng * (BN / 2) + j * 16 + 4 * q) * 2) = make_uint2(lo, hi);
                    }
                }
            }
        }
    };
    with_count<WM>(__builtin_amdgcn_readfirstlane((rows + 63) / 64), k_walk);
    __syncthreads();
    if constexpr (UP) {
        constexpr int CH = BN / 16;
        for (int idx = tid; idx < rows * CH; idx += 512) {
            const int row = idx / CH, ch = idx % CH;
            *(uint4*)(g.out + ((int64_t)row0 + row) * g.ldo + n0 + ch * 16) = *(const uint4*)(ring + row * OSTR + ch * 16);
        }
    } else {
        store_tile_bf16<BM, BN, OSTR, 512, true>(ring, g.out, g.ldo, row0, rows, n0);
    }
}

template <bool UP>
static void launch_mx(const moe_shape_t& s, GemmArgs a, int N, hipStream_t stream)
{
    const bool wide = !UP && N % 256 == 0;             // down: 256-wide n-blocks where d allows
    const bool few = tile_rows(s) == 16;
    a.n_blocks = few && !UP ? (N + 255) / 256 : N / (wide ? 256 : 128);
    const unsigned grid = (unsigned)launch_blocks(a);
    // scale rows in 16-byte words: of both operands, of routed and shared groups
    const uintptr_t at = (uintptr_t)a.As | (uintptr_t)a.B1s | (uintptr_t)a.B3s | (uintptr_t)a.S1s | (uintptr_t)a.S3s;
    const bool sc16 = ((at | (uintptr_t)a.ldas | (uintptr_t)(a.K_r / 32) | (uintptr_t)(a.S1s ? a.K_s / 32 | a.nkb_s : 0)) & 15) == 0;
    if (few) mx_gemm_stream_kernel<UP><<<grid, 1024, 0, stream>>>(a);
    else if (UP || !wide) {
        if (sc16) mx_gemm_kernel<UP, 128, true><<<grid, 512, 0, stream>>>(a);
        else mx_gemm_kernel<UP, 128, false><<<grid, 512, 0, stream>>>(a);
    } else if constexpr (!UP) {
        if (sc16) mx_gemm_kernel<false, 256, true><<<grid, 512, 0, stream>>>(a);
        else mx_gemm_kernel<false, 256, false><<<grid, 512, 0, stream>>>(a);
    }
}

static GemmArgs mx_args(const moe_shape_t& s, const Workspace& ws, int e_base)
{
    GemmArgs a = {};
    a.e_base = e_base;
    a.tiles = ws.tiles;
    a.ntiles = ws.sync;
    a.max_tiles = (int)ws.max_tiles;
    a.E = (int)s.E;
    a.group_m = tile_rows(s) == 16 ? 0 : 2;
    return a;
}

hipError_t launch_up_gemm_mx(const moe_shape_t& s, const void* W1, const void* W3, const void* W1s, const void* W3s,
                             const void* S1, const void* S3, const void* S1s, const void* S3s, const Workspace& ws,
                             hipStream_t stream, int e_base, int n_shared)
{
    GemmArgs up = mx_args(s, ws, e_base);
    up.row_token = ws.row_token;
    up.A = ws.xq;
    up.As = (const float*)ws.xe;
    up.lda = s.d;
    up.ldas = s.d / 32;
    up.B1 = (const uint8_t*)W1;
    up.B3 = (const uint8_t*)W3;
    up.B1s = (const float*)W1s;
    up.B3s = (const float*)W3s;
    up.S1 = (const uint8_t*)S1;
    up.S3 = (const uint8_t*)S3;
    up.S1s = (const float*)S1s;
    up.S3s = (const float*)S3s;
    up.ld_s = s.d;
    up.nkb_s = (int)(s.d / 32);
    up.out = (uint8_t*)ws.h;
    up.outs = (float*)ws.he;
    up.ldo = ws.inter_max;
    up.ldos = ws.inter_max / 32;
    up.N_r = (int)s.inter;
    up.N_s = n_shared;
    up.K_r = up.K_s = (int)s.d;
    launch_mx<true>(s, up, (int)ws.inter_max, stream);
    return hipGetLastError();
}

hipError_t launch_down_gemm_mx(const moe_shape_t& s, const void* W2, const void* W2s, const void* S2, const void* S2s,
                               const Workspace& ws, hipStream_t stream, int e_base, int n_shared)
{
    GemmArgs dn = mx_args(s, ws, e_base);
    dn.A = (const uint8_t*)ws.h;
    dn.As = (const float*)ws.he;
    dn.lda = ws.inter_max;
    dn.ldas = ws.inter_max / 32;
    dn.B1 = (const uint8_t*)W2;
    dn.B1s = (const float*)W2s;
    dn.S1 = (const uint8_t*)S2;
    dn.S1s = (const float*)S2s;
    dn.ld_s = n_shared;
    dn.nkb_s = n_shared / 32;
    dn.out = (uint8_t*)ws.y_rows;
    dn.ldo = s.d;
    dn.N_r = dn.N_s = (int)s.d;
    dn.K_r = (int)s.inter;
    dn.K_s = n_shared;
    launch_mx<false>(s, dn, (int)s.d, stream);
    return hipGetLastError();
}

}  // namespace moe
