// mx.hip -- the microscaled formats on their own: quantisation of a matrix and reading it back.
//
// Both are one pass over dense rows whose length is a multiple of 32, so a matrix is a flat run of groups.
// A lane holds eight elements of a group, four lanes the group: loads and stores are whole 16-byte (bf16)
// or 32-byte (fp32) vectors a lane, the group's maximum takes two DPP moves, and no element is read twice.
// HBM bounds both: a 2048 x 7168 bf16 matrix becomes MXFP4 in 8.0 us (37 MB read and written, 4.6 TB/s) and is read
// back in 7.6 us (4.9 TB/s), where a large device copy reaches 4.8; 64 rows take 2.5 us, a launch.
#include "mx.h"

namespace moe {

template <bool BF16> struct MxVec;
template <> struct MxVec<true> {
    uint4 r;
    __device__ __forceinline__ void load(const void* p, int64_t i) { r = ((const uint4*)p)[i]; }
    __device__ __forceinline__ void get(float (&v)[8]) const { bf16x8_to_f32(r, v); }
};
template <> struct MxVec<false> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t i)
    {
        a = ((const float4*)p)[2 * i];
        b = ((const float4*)p)[2 * i + 1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// n8: vectors of eight elements (a multiple of four).  A group with an infinity or NaN gets scale 255 and
// zero codes.
template <bool FP4, bool BF16>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, int64_t n8, uint8_t* __restrict__ q,
                                                          uint8_t* __restrict__ scales)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;                               // whole groups of four lanes leave together
    MxVec<BF16> r;
    r.load(x, i);
    float v[8];
    r.get(v);
    const uint32_t c = mx_scale_code<FP4>(quad_max(mx_amax8(v)));
    if constexpr (FP4) ((uint32_t*)q)[i] = c == 255u ? 0u : mx_pack_fp4(v, c);
    else ((uint2*)q)[i] = c == 255u ? make_uint2(0u, 0u) : mx_pack_fp8(v, c);
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)c;
}

// Reading back: code * 2^(c - 127) in fp32 (exact: at most four significant bits), rounded to bf16 where that
// is asked for (exact too, but for MXFP8 values under 2^-133); scale 255 gives NaN.
template <bool FP4, bool BF16>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales,
                                                            int64_t n8, void* __restrict__ out)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const uint32_t c = scales[i >> 2];
    const float s = __uint_as_float(c << 23);
    f32x2_t p[4];
    if constexpr (FP4) {
        const uint32_t w = ((const uint32_t*)q)[i];
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    } else {
        const uint2 w = ((const uint2*)q)[i];
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.x, s, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.x, s, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.y, s, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w.y, s, true);
    }
    if (c == 255u) {
#pragma unroll
        for (int e = 0; e < 4; e++) p[e].x = p[e].y = __uint_as_float(0x7FC00000u);
    }
    if constexpr (BF16) {
        ((uint4*)out)[i] = make_uint4(f32x2_to_bf16x2(p[0].x, p[0].y), f32x2_to_bf16x2(p[1].x, p[1].y),
                                      f32x2_to_bf16x2(p[2].x, p[2].y), f32x2_to_bf16x2(p[3].x, p[3].y));
    } else {
        ((float4*)out)[2 * i] = make_float4(p[0].x, p[0].y, p[1].x, p[1].y);
        ((float4*)out)[2 * i + 1] = make_float4(p[2].x, p[2].y, p[3].x, p[3].y);
    }
}

hipError_t launch_quantize_mx(int64_t n, bool fp4, bool bf16, const void* x, uint8_t* q, uint8_t* scales,
                              hipStream_t stream)
{
    const int64_t n8 = n / 8;
    const unsigned grid = (unsigned)((n8 + 255) / 256);
    if (fp4 && bf16) mx_quantize_kernel<true, true><<<grid, 256, 0, stream>>>(x, n8, q, scales);
    else if (fp4) mx_quantize_kernel<true, false><<<grid, 256, 0, stream>>>(x, n8, q, scales);
    else if (bf16) mx_quantize_kernel<false, true><<<grid, 256, 0, stream>>>(x, n8, q, scales);
    else mx_quantize_kernel<false, false><<<grid, 256, 0, stream>>>(x, n8, q, scales);
    return hipGetLastError();
}

hipError_t launch_dequantize_mx(int64_t n, bool fp4, bool bf16, const uint8_t* q, const uint8_t* scales, void* out,
                                hipStream_t stream)
{
    const int64_t n8 = n / 8;
    const unsigned grid = (unsigned)((n8 + 255) / 256);
    if (fp4 && bf16) mx_dequantize_kernel<true, true><<<grid, 256, 0, stream>>>(q, scales, n8, out);
    else if (fp4) mx_dequantize_kernel<true, false><<<grid, 256, 0, stream>>>(q, scales, n8, out);
    else if (bf16) mx_dequantize_kernel<false, true><<<grid, 256, 0, stream>>>(q, scales, n8, out);
    else mx_dequantize_kernel<false, false><<<grid, 256, 0, stream>>>(q, scales, n8, out);
    return hipGetLastError();
}

}  // namespace moe
