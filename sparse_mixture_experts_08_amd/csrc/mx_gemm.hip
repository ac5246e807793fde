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
// ---------------------------------------------------------------------------------------------------
template <bool UP>
__global__ __launch_bounds__(1024, 4) void mx_gemm_stream_kernel(GemmArgs g)
{
    constexpr int NW = 16, NT = 64 * NW, FW = UP ? 8 : 16, BN = NW * FW, D = 4;
    constexpr int XK = UP ? 7168 : 4096, XSTR = XK + 16;               // whole rounds of D units
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
// 128- and 256-row tiles: eight wavefronts as 2 (rows) x 4 (features), operands and scales staged through LDS
// by direct-to-LDS loads.  A K stage is 128 elements: 128 bytes of every activation row, 64 of every weight
// row, and four scale bytes of each.  The 16-row blocks of a tile alternate between the two row groups of
// wavefronts, so a tile that is not full still spreads over both.  A stage's LDS: BM rows of 128 bytes, NB rows
// of 64 (both swizzled by row: see gemm.h), 512 scale words.
// ---------------------------------------------------------------------------------------------------
template <bool UP, int BM, int BN, int NSTG>
__global__ __launch_bounds__(512, 2) void mx_gemm_kernel(GemmArgs g)
{
    constexpr int NB = UP ? 2 * BN : BN;               // weight rows per stage
    constexpr int WM = BM / 32, WN = BN / 64;          // 16-row and 16-feature blocks per wavefront
    constexpr int PA = BM / 64, PB = NB / 128;         // 1-KB loads per wavefront and stage: activations, weights
    constexpr int NL = PA + PB + 1;                    // ... and one load of scales
    constexpr int STAGE = BM * 128 + NB * 64;
    static_assert(BM == 128 || BM == 256, "128- or 256-row tiles");
    static_assert(!UP || BN == 128, "a wavefront's 32 features of h are one group");
    static_assert(BM / 64 <= 4 && NB / 64 <= 4, "wavefronts 0-3 copy activation scales, 4-7 weight scales");
    static_assert((NSTG - 1) * NL < 64, "vmcnt range");
    constexpr int OSTR = (UP ? BN : BN * 2) + 16;      // epilogue: padded LDS row of the output tile
    constexpr int RING = NSTG * STAGE > BM * OSTR ? NSTG * STAGE : BM * OSTR;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[RING];
    __shared__ __attribute__((aligned(256))) uint32_t scl[NSTG][512];
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
    const int mg = wave >> 2, ng = wave & 3;           // row group, feature group
    const int r16 = lane & 15, q = lane >> 4;
    const MxGroup m = mx_group<UP>(g, grp, shared, N, K);

    // rows past the tile's end repeat its first row (valid memory; computed or skipped, never stored)
    if (tid < BM) s_tok[tid] = UP ? g.row_token[row0 + (tid < rows ? tid : 0)] : row0 + (tid < rows ? tid : 0);
    __syncthreads();

    // Sources, fixed over the K walk (32-bit offsets: the host keeps every operand under 4 GB).  Lane l of a load
    // writes 16-byte chunk l % 8 of row l / 8 (activations) or l % 4 of row l / 4 (weights) and so reads the
    // logical chunk that the swizzle keeps there.
    uint32_t offA[PA], offB[PB];
#pragma unroll
    for (int p = 0; p < PA; p++) {
        const int row = (p * 8 + wave) * 8 + (lane >> 3);
        offA[p] = (uint32_t)s_tok[row] * (uint32_t)g.lda + (swzr<128>(row, lane & 7) - row * 128);
    }
#pragma unroll
    for (int p = 0; p < PB; p++) {
        const int row = (p * 8 + wave) * 16 + (lane >> 2);             // UP: rows BN .. are W3's
        offB[p] = (uint32_t)(n0 + (UP ? row % BN : row)) * (uint32_t)m.ldb + (swzr<64>(row, lane & 3) - row * 64);
    }
    // Scale words in the order the wavefronts read them: activations of row group mg at mg BM / 2 + 64 v + 4 r16 +
    // e = row 16 (2 (4 v + e) + mg) + r16; weights of feature group ng, matrix by matrix, at 16 WN ng + WN r16 + e
    // = feature 16 WN ng + 16 e + r16.
    uint32_t offS = 0;
    const uint8_t* baseS = bytes(g.As);
    if (wave < 4) {
        const int p = (wave * 64 + lane) % BM, rem = p % (BM / 2);     // BM = 128: wavefronts 2, 3 repeat 0, 1
        const int row = 16 * (2 * (4 * (rem / 64) + rem % 4) + p / (BM / 2)) + (rem % 64) / 4;
        offS = (uint32_t)s_tok[row] * (uint32_t)g.ldas;
    } else {
        const int p = ((wave - 4) * 64 + lane) % NB, f = p % BN, rem = f % (16 * WN);
        const int row = f - rem + 16 * (rem % WN) + rem / WN;
        offS = (uint32_t)(n0 + row) * (uint32_t)m.nkb;
        baseS = UP && ((wave - 4) * 64) % NB >= BN ? m.W3s : m.W1s;    // BN is a multiple of 64: wave-uniform
    }

    const int nstages = K / 128;
    const int kshift = (nb * g.krot) % nstages;
    const uint32_t ring0 = lds_addr(ring), scl0 = lds_addr(&scl[0][0]);
    auto issue = [&](int buf, int s) {
        const int ks = s + kshift >= nstages ? s + kshift - nstages : s + kshift;
        const uint32_t dst = ring0 + buf * STAGE + wave * 1024;
#pragma unroll
        for (int p = 0; p < PA; p++) dma16(g.A + (int64_t)ks * 128, offA[p], dst + p * 8192);
#pragma unroll
        for (int p = 0; p < PB; p++)
            dma16((UP && p * 128 >= BN ? m.W3 : m.W1) + (int64_t)ks * 64, offB[p], dst + BM * 128 + p * 8192);
        dma4(baseS + (int64_t)ks * 4, offS, scl0 + (buf * 512 + wave * 64) * 4);
    };

    f32x4 acc1[WM][WN], acc3[WM][UP ? WN : 1];
#pragma unroll
    for (int i = 0; i < WM; i++) {
#pragma unroll
        for (int j = 0; j < WN; j++) acc1[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < (UP ? WN : 1); j++) acc3[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    // 16-row blocks of this wavefront that hold tile rows (wave-uniform): i with 16 (2 i + mg) < rows
    const int nrb = __builtin_amdgcn_readfirstlane(max(0, min(WM, ((rows + 15) / 16 - mg + 1) / 2)));

    auto k_walk = [&](auto nb_tag) {
        constexpr int NR = decltype(nb_tag)::value;
#pragma unroll
        for (int t = 0; t < NSTG; t++) issue(t, min(t, nstages - 1));
        wait_vmcnt<(NSTG - 1) * NL>();
        lds_barrier();
        int buf = 0;
        for (int s = 0; s < nstages; s++) {
            const uint8_t* sa = ring + buf * STAGE;
            const uint8_t* sb = sa + BM * 128;
            const uint32_t* sc = scl[buf];
            if constexpr (NR > 0) {
                i32x8 b1[WN], b3[UP ? WN : 1];
                uint32_t s1[WN], s3[UP ? WN : 1], as[WM];
                auto wfrag = [&](int row) {
                    const i32x4 lo = *(const i32x4*)(sb + swzr<64>(row, q));
                    return (i32x8){lo.x, lo.y, lo.z, lo.w, 0, 0, 0, 0};
                };
#pragma unroll
                for (int j = 0; j < WN; j++) {
                    b1[j] = wfrag(ng * 16 * WN + 16 * j + r16);
                    s1[j] = sc[256 + ng * 16 * WN + r16 * WN + j] >> (8 * q);
                    if constexpr (UP) {
                        b3[j] = wfrag(BN + ng * 16 * WN + 16 * j + r16);
                        s3[j] = sc[256 + BN + ng * 16 * WN + r16 * WN + j] >> (8 * q);
                    }
                }
#pragma unroll
                for (int i = 0; i < NR; i++) as[i] = sc[mg * (BM / 2) + 64 * (i / 4) + 4 * r16 + i % 4] >> (8 * q);
#pragma unroll
                for (int i = 0; i < NR; i++) {
                    const int row = 16 * (2 * i + mg) + r16;
                    const i32x4 lo = *(const i32x4*)(sa + swzr<128>(row, q));
                    const i32x4 hi = *(const i32x4*)(sa + swzr<128>(row, 4 + q));
                    const i32x8 a = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int j = 0; j < WN; j++) {
                        acc1[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b1[j], a, acc1[i][j], 4, 0, 0, (int)s1[j], 0, (int)as[i]);
                        if constexpr (UP)
                            acc3[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b3[j], a, acc3[i][j], 4, 0, 0, (int)s3[j], 0, (int)as[i]);
                    }
                }
            }
            if (s + 1 < nstages) {
                wait_vmcnt<(NSTG - 2) * NL>();         // stage s + 1 has landed
                lds_barrier();                         // ... for every wavefront, and stage s is read
                issue(buf, min(s + NSTG, nstages - 1)); // past the end: the last stage again (never read)
                buf = buf + 1 == NSTG ? 0 : buf + 1;
            }
        }
    };
    with_count<WM>(nrb, k_walk);
    wait_vmcnt<0>();                                   // no load may still target this block's LDS
    lds_barrier();

    if constexpr (UP) {
        // h of a token's 32 features (this wavefront's) lies on the four lanes r16 + 16 q, eight values each
#pragma unroll
        for (int i = 0; i < WM; i++) {
            const int row = 16 * (2 * i + mg) + r16;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float gg = acc1[i][e / 4][e % 4], uu = acc3[i][e / 4][e % 4];
                round_bf16x2(gg, uu);
                v[e] = round_bf16(silu_mul_fast(gg, uu));
            }
            uint32_t am = mx_amax8(v);
            am = max(am, (uint32_t)__shfl_xor((int)am, 16, 64));
            am = max(am, (uint32_t)__shfl_xor((int)am, 32, 64));
            const uint32_t c = mx_scale_code<false>(am);
            const uint2 p = c == 255u ? make_uint2(0u, 0u) : mx_pack_fp8(v, c);
            *(uint32_t*)(ring + row * OSTR + ng * 32 + 4 * q) = p.x;
            *(uint32_t*)(ring + row * OSTR + ng * 32 + 16 + 4 * q) = p.y;
            if (q == 0 && row < rows) ((uint8_t*)g.outs)[((int64_t)row0 + row) * g.ldos + n0 / 32 + ng] = (uint8_t)c;
        }
        __syncthreads();
        constexpr int CH = BN / 16;
        for (int idx = tid; idx < BM * CH; idx += 512) {
            const int row = idx / CH, ch = idx % CH;
            if (row < rows)
                *(uint4*)(g.out + ((int64_t)row0 + row) * g.ldo + n0 + ch * 16) = *(const uint4*)(ring + row * OSTR + ch * 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < WM; i++)
#pragma unroll
            for (int j = 0; j < WN; j++) {
                const uint32_t lo = f32x2_to_bf16x2(acc1[i][j][0], acc1[i][j][1]);
                const uint32_t hi = f32x2_to_bf16x2(acc1[i][j][2], acc1[i][j][3]);
                *(uint2*)(ring + (16 * (2 * i + mg) + r16) * OSTR + (ng * 16 * WN + j * 16 + 4 * q) * 2) = make_uint2(lo, hi);
            }
        __syncthreads();
        store_tile_bf16<BM, BN, OSTR, 512, true>(ring, g.out, g.ldo, row0, rows, n0);
    }
}

template <bool UP>
static void launch_mx(const moe_shape_t& s, GemmArgs a, int N, hipStream_t stream)
{
    const int bm = tile_rows(s);
    const bool wide = !UP && N % 256 == 0;             // down: 256-wide n-blocks where d allows
    a.n_blocks = bm == 16 && !UP ? (N + 255) / 256 : N / (wide ? 256 : 128);
    const unsigned grid = (unsigned)launch_blocks(a);
    if (bm == 16) mx_gemm_stream_kernel<UP><<<grid, 1024, 0, stream>>>(a);
    else if constexpr (UP) {
        if (bm == 128) mx_gemm_kernel<true, 128, 128, 4><<<grid, 512, 0, stream>>>(a);
        else mx_gemm_kernel<true, 256, 128, 3><<<grid, 512, 0, stream>>>(a);
    } else if (wide) {
        if (bm == 128) mx_gemm_kernel<false, 128, 256, 4><<<grid, 512, 0, stream>>>(a);
        else mx_gemm_kernel<false, 256, 256, 3><<<grid, 512, 0, stream>>>(a);
    } else {
        if (bm == 128) mx_gemm_kernel<false, 128, 128, 4><<<grid, 512, 0, stream>>>(a);
        else mx_gemm_kernel<false, 256, 128, 3><<<grid, 512, 0, stream>>>(a);
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
    a.group_m = tile_rows(s) == 16 ? 0 : 4;
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
