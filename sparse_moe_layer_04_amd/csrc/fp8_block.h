// Device helpers and launchers of the 128-block 8-bit operators.
#pragma once

#include "moe_internal.h"

namespace moe {

// blocks of 128 along a side of n (64-bit: n + 127 passes 2^31 for the longest)
__host__ __device__ constexpr long long block_count(long long n) { return (n + 127) / 128; }
static_assert(block_count(0x7fffffff) == 1ll << 24, "the longest side");

// 2^X for X in [-126, 127]
__device__ __forceinline__ float pow2(int X) { return __uint_as_float((uint32_t)(X + 127) << 23); }

// |v|, 0 where v is not finite
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;
}

// the least X with amax <= 448 * 2^X, within [-126, 120]; 0 for amax = 0
// (a subnormal amax has exponent field 0 and takes the lower limit)
__device__ __forceinline__ int block_exponent(float amax) {
    if (!(amax > 0.0f)) return 0;
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127;
    return max(e - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7), -126);
}

// four E4M3 codes of v * inv (|v * inv| <= 448; nearest, ties to even), NaN
// codes where v is not finite
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d, float inv) {
    const float nan = __builtin_nanf("");
    const float inf = __builtin_inff();
    a = fabsf(a) < inf ? a * inv : nan;
    b = fabsf(b) < inf ? b * inv : nan;
    c = fabsf(c) < inf ? c * inv : nan;
    d = fabsf(d) < inf ? d * inv : nan;
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    return (uint32_t)r;
}

// two fp32 values as bf16 (nearest, ties to even, NaN kept), a in the low half
__device__ __forceinline__ uint32_t bf16_pack2(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// lanes 0-31: a of lane l and of lane l + 32; lanes 32-63: b of lane l - 32
// and of lane l
__device__ __forceinline__ u32x2 swap_halves(uint32_t a, uint32_t b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    return u32x2{r[0], r[1]};
}

// maximum of v >= 0 over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float row16_max(float v) {
#define MOE_DPP_MAX(CTRL)                                                                   \
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, \
                                                            0xf, false)));
    MOE_DPP_MAX(0xB1)    // quad_perm [1,0,3,2]
    MOE_DPP_MAX(0x4E)    // quad_perm [2,3,0,1]
    MOE_DPP_MAX(0x141)   // row_half_mirror
    MOE_DPP_MAX(0x140)   // row_mirror
#undef MOE_DPP_MAX
    return v;
}

// Inclusive sum over the wave's lanes
__device__ __forceinline__ int wave_scan(int x, int lane) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
    }
    return x;
}

// silu(clamp(g)) * clamp(u), the expert FFN's activation (comparisons, so
// that a NaN passes the clamps)
__device__ __forceinline__ float clamped_swiglu(float g, float u, float L, int mode) {
    g = g > L ? L : g;
    if (mode == MOE_CLAMP_SYMMETRIC) g = g < -L ? -L : g;
    u = u > L ? L : u;
    u = u < -L ? -L : u;
    return g / (1.0f + __expf(-g)) * u;
}

// ----------------------------------------------------------------- host -----
hipError_t launch_quant_rows_fp8_block(const void* a, int in_dtype, long long rows, int K,
                                       uint8_t* codes, float* scales, hipStream_t stream);
hipError_t launch_quant_matrix_fp8_block(const void* w, int in_dtype, int G, int N, int K,
                                         uint8_t* codes, float* scales, hipStream_t stream);

struct Fp8GemmArgs {
    const uint8_t* a;        // [rows, K] E4M3 codes
    const float* as;         // [rows, ceil(K / 128)]
    const int32_t* offsets;  // [G + 1] device
    int G, rows, K;
    int N;                   // weight rows a group (SwiGLU: features)
    const uint8_t* w1;       // [G, N, K] E4M3 codes
    const uint8_t* w2;       // (SwiGLU: the up matrices)
    const float* s1;         // [G, ceil(N / 128), ceil(K / 128)]
    const float* s2;
    float clamp_limit;
    int clamp_mode;
    void* out;               // [rows, N] fp32 or bf16; SwiGLU: E4M3 codes of h
    float* out_scale;        // SwiGLU: [rows, ceil(N / 128)]
};
enum Fp8Epilogue : int { FP8_OUT_BF16 = 0, FP8_OUT_F32 = 1, FP8_SWIGLU = 2 };
hipError_t launch_grouped_gemm_fp8_block(int epilogue, const Fp8GemmArgs& g, hipStream_t stream);

}  // namespace moe
