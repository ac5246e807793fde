// gemm.h -- what the grouped expert GEMMs share: their arguments, the block -> work mapping, the SwiGLU
// epilogue's arithmetic and the direct-to-LDS staging.
#pragma once

#include "moe_common.h"

namespace moe {

struct GemmArgs {
    const int4* tiles;        // tile list
    const int32_t* ntiles;    // number of valid tiles
    const int32_t* row_token; // up: sorted row -> token (A row)
    const uint8_t* A;         // up: x or its E4M3 codes; down: h
    const float* As;          // fp8: scales of A rows per 128-K block ([rows, K/128])
    int64_t lda;              // bytes between A rows
    int64_t ldas;             // floats between rows of As
    const uint8_t* B1;        // routed weights (up: W1, down: W2) [experts e_base.., N, K]
    const uint8_t* B3;        // up: W3
    const float* B1s;         // fp8 block scales [E, N/128, K/128]
    const float* B3s;
    const uint8_t* S1;        // shared-expert weights [N_s rows of ld_s elements, K_s used]
    const uint8_t* S3;
    const float* S1s;
    const float* S3s;
    uint8_t* out;             // up: h; down: y_rows
    float* outs;              // up with fp8: scales of h [rows, inter_max/128]
    int64_t ldo;              // elements between output rows
    int64_t ldos;             // floats between rows of outs
    int E;                    // group E is the shared expert
    int e_base;               // expert held at index 0 of B1/B3 (and their scales)
    int N_r, N_s;             // output features: routed / shared
    int K_r, K_s;             // reduction length: routed / shared
    int n_blocks;             // n-blocks per tile (over the larger N)
    int64_t ld_s;             // elements between shared weight rows (a slice of a wider expert)
    int nkb_s;                // fp8: scale blocks between shared scale rows
    int max_tiles;
    int krot;                 // K-stage rotation per n-block (0: every block walks K from stage 0)
    int group_m;              // 0: block b -> (tile b / n_blocks, n-block b % n_blocks); else the XCD-aware
                              // grouped order below, with group_m tiles per group
};

__device__ __forceinline__ float silu_mul(float g, float u)
{
    const float sig = 1.0f / (1.0f + expf(-g));
    return (g * sig) * u;
}

// silu(g) * u for an h that is rounded to bf16 (the bf16 and fp8 layers): the sigmoid from the hardware
// base-2 exponential and reciprocal (v_exp_f32, v_rcp_f32, each within about an ulp), five instructions
// where expf and the IEEE division take about 25.  Its error, under 1e-6 relative, is far below a bf16
// ulp (2^-8): over normally distributed g an emulation moves 1 to 2 in 10^5 of the rounded h values by
// one bf16 ulp against the IEEE form.  The fp32 layer keeps silu_mul.  In the large-tile GEMMs the
// epilogue runs with the matrix pipe idle, so its cost adds to the kernel's time.
__device__ __forceinline__ float silu_mul_fast(float g, float u)
{
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504088896341f);   // exp(-g)
    const float sig = __builtin_amdgcn_rcpf(1.0f + e);
    return (g * sig) * u;
}

// block -> (tile, n-block); false when the block has no work.  group_m == 0 (decode-sized tiles):
// consecutive blocks walk one tile's n-blocks.  Otherwise the work list is cut into groups of group_m
// consecutive tiles x all n-blocks, walked n-block by n-block with the group's tiles fastest, and the
// groups are dealt round-robin to the 8 XCDs (block b runs on XCD b % 8; XCD x takes groups x, x + 8,
// x + 16, ..., one after the other).  Blocks that run together on one XCD share A rows (same tile) and
// weight panels (same expert, n-block) in that XCD's L2, and every XCD gets a like share of hot, cold and
// shared-expert tiles: cut into 8 contiguous ranges instead, the list gave one XCD all 16 shared tiles of
// the 4096-token layer (about a quarter more work than the others) and the skewed layer's XCDs 5-6 % more
// or less than their mean.  launch_blocks() is the grid this needs.
__device__ __forceinline__ bool block_work(const GemmArgs& g, int& tile, int& nb)
{
    const int bid = blockIdx.x;
    const int nt = *g.ntiles;
    if (g.group_m == 0) {
        tile = bid / g.n_blocks;
        nb = bid % g.n_blocks;
        return tile < nt;
    }
    const int items = g.group_m * g.n_blocks;          // work items of a full group
    const int j = bid >> 3;                            // the block's place in its XCD's list
    const int c = (bid & 7) + 8 * (j / items), r = j % items;
    if (c * g.group_m >= nt) return false;
    const int gm = min(g.group_m, nt - c * g.group_m); // the last group may be short
    if (r >= gm * g.n_blocks) return false;
    nb = r / gm;
    tile = c * g.group_m + r % gm;
    return true;
}

// Grid of a grouped-GEMM launch: enough blocks for max_tiles tiles under block_work's mapping.
static int64_t launch_blocks(const GemmArgs& a)
{
    if (a.group_m == 0) return ((int64_t)a.n_blocks * a.max_tiles + 7) / 8 * 8;
    const int64_t groups = (a.max_tiles + a.group_m - 1) / a.group_m;
    return 8 * ((groups + 7) / 8) * a.group_m * a.n_blocks;
}

// ---------------------------------------------------------------------------------------------------
// Machinery of the direct-to-LDS forms below.  K stages are copied global -> LDS by the direct-to-LDS
// load (global_load_lds_dwordx4: a wavefront's 64 lanes write 1 KB at M0 + 16 * lane), so staging uses
// no registers, no LDS store instructions and no per-load vector-ALU work: each lane's source is a
// block-uniform base in SGPRs (moved by the K stage) plus a 32-bit offset fixed for the whole K walk.
// The loads are issued from asm, so the compiler knows of no load into LDS and schedules fragment reads
// freely; an explicit vmcnt wait and barrier per stage order the reads after the loads of their stage.
//
// LDS row layout: 16-byte chunk c of row r stored at chunk c ^ f(r), f(r) = (r ^ (r >> 3 & 1)) & 7 for
// 128-byte rows, ((r >> 1) ^ (r >> 3)) & 3 for 64-byte rows: a fragment read (lanes 0..31: 32
// consecutive rows, one chunk) hits distinct banks for any 8 or 16 consecutive lanes, and f is unchanged
// by adding 16 (resp. 32) rows.  The loads apply the swizzle on the source side (lane l writes stored
// chunk l % (RB / 16) of row l / (RB / 16), so it reads the logical chunk that belongs there).
// Rows past the tile's end load the tile's first row (valid memory); their results are never stored.
// ---------------------------------------------------------------------------------------------------
typedef float f32x16 __attribute__((ext_vector_type(16)));
template <int N> struct IntC {
    static constexpr int value = N;
};

// f(IntC<n>{}) for a runtime n in [0, N] (n outside: f(IntC<0>{})).
template <int N, typename F> __device__ __forceinline__ void with_count(int n, F&& f)
{
    if constexpr (N == 0) {
        f(IntC<0>{});
    } else {
        if (n == N) f(IntC<N>{});
        else with_count<N - 1>(n, f);
    }
}

template <int N> __device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Barrier without the vmcnt(0) that __syncthreads implies: loads into the other ring buffers stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int RB> __device__ __forceinline__ int swzr(int row, int chunk)
{
    if constexpr (RB == 128) return row * 128 + ((chunk ^ ((row ^ (row >> 3 & 1)) & 7)) << 4);
    else return row * 64 + ((chunk ^ (((row >> 1) ^ (row >> 3)) & 3)) << 4);
}

__device__ __forceinline__ uint32_t lds_addr(const void* p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// One direct-to-LDS load: lane l copies 16 bytes from sbase + voff to LDS address lds + 16 l.  M0 carries
// the LDS address and is written here (one wait state before the load uses it); nothing else in the
// kernels that use this keeps a value in M0.  No memory clobber: the load writes a ring buffer that no
// LDS access nearby touches, and as a volatile asm it keeps its place relative to the barrier asm.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const uint8_t* sbase, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase), "s"(lds)
                 : "m0");
}
// The 4-byte form: lane l copies 4 bytes from sbase + voff to LDS address lds + 4 l.
__device__ __forceinline__ void dma4(const uint8_t* sbase, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(sbase), "s"(lds)
                 : "m0");
}
#pragma clang diagnostic pop

// Coalesced store of a block's bf16 output tile: the wavefronts have written it row-major into LDS (row
// stride OSTR bytes, padded so the two row groups of one LDS write fall on different banks); every
// thread then copies 16-byte chunks of rows < rows to out (row0 + row, col0 ..), ldo elements apart.
// Against per-lane 2-byte global stores straight from the accumulators this writes whole lines (and
// against 8-byte stores straight from the fp8 kernel's accumulators, 32 contiguous bytes a row: fp8 down
// GEMM 4.83 -> 5.35 ms).  NTS: stores with the non-temporal hint, for the down GEMMs' expert-output rows,
// which only the combine reads, after the whole GEMM (prefill down GEMM 1.795 -> 1.695 ms, fp8 down GEMM
// 4.77 -> 4.68 ms, skewed down GEMM 0.3 % slower).
template <int BM, int OC, int OSTR, int NT, bool NTS = false>
__device__ __forceinline__ void store_tile_bf16(const uint8_t* tile, uint8_t* out, int64_t ldo, int row0, int rows,
                                                int col0)
{
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    constexpr int CH = OC * 2 / 16;                    // 16-byte chunks per row
    for (int idx = threadIdx.x; idx < BM * CH; idx += NT) {
        const int row = idx / CH, ch = idx % CH;
        if (row < rows) {
            u32x4_t* dst = (u32x4_t*)(out + (((int64_t)row0 + row) * ldo + col0 + ch * 8) * 2);
            const u32x4_t v = *(const u32x4_t*)(tile + row * OSTR + ch * 16);
            if constexpr (NTS) __builtin_nontemporal_store(v, dst);
            else *dst = v;
        }
    }
}

}  // namespace moe
