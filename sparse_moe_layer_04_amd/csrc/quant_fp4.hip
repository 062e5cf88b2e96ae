// MXFP4 quantisation of rows: E2M1 codes with one power-of-two scale for each
// 32 values,
//   X = floor(log2(max |v|)) - 2 in [-127, 127] (0 for zeros), scale byte
//   X + 127; code = E2M1(v / 2^X), nearest, ties to even, saturating at +-6;
// a block that holds an infinity or NaN gets the scale byte 255 (NaN).
// v / 2^X is exact (a power of two; where it is subnormal the code is 0 on
// either side of its rounding).
//
// The rows are one run of blocks (K is a multiple of 32), whatever K is.  Four
// lanes take a block, eight values each (so that a wave's loads cover whole
// lines), a thread kU blocks with their loads in flight together.
//
// Bound: HBM, 2.53 bytes a bf16 value: 49152 x 4096 84 us, 6.1 TB/s; 8191 x
// 4064 fp32 25 us (6.0, half of it from the cache).  A lane a block (16 bytes
// of each of 64 lines a load) and a conversion in software took 103 and 29.
// Loads past the caches: 78 where nothing is found there, but 32 for 25 and 55
// for 48 behind a kernel that wrote the rows.
#include "fp4.h"

namespace moe {
namespace {

constexpr int kU = 4;

// maximum over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));
}

template <bool F32>
__global__ __launch_bounds__(256) void quant_mxfp4_kernel(const void* __restrict__ a,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales,
                                                          long long blocks) {
    const long long first = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * (64 * kU) +
                            (threadIdx.x >> 2);
    const int part = threadIdx.x & 3;
    u32x4 w[kU][F32 ? 2 : 1];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const long long b = first + 64 * u;
        const u32x4* src = (const u32x4*)((const uint8_t*)a +
                                          (size_t)(b < blocks ? b : blocks - 1) * (F32 ? 128 : 64));
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) w[u][i] = src[(F32 ? 2 : 1) * part + i];
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const long long b = first + 64 * u;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (F32) v[i] = __uint_as_float(w[u][i >> 2][i & 3]);
            else v[i] = __uint_as_float(i & 1 ? w[u][0][i >> 1] & 0xffff0000u
                                              : w[u][0][i >> 1] << 16);
        }
        uint32_t top = 0;                  // |v| as bits: infinities and NaN are the largest
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        top = quad_max(top);
        // (a subnormal maximum has exponent field 0: X = -127 as for all below 2^-124)
        const int X = top == 0 ? 0 : max((int)(top >> 23) - 129, -127);
        const bool bad = top >= 0x7f800000u;
        const float inv = __uint_as_float((uint32_t)(127 - X) << 23);  // 2^-X: X in [-127, 126]
        // (the hardware's conversion rounds to nearest, ties to even, and saturates)
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * inv, v[1] * inv, 1.0f, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * inv, v[3] * inv, 1.0f, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * inv, v[5] * inv, 1.0f, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * inv, v[7] * inv, 1.0f, 3);
        if (b < blocks) {
            *(uint32_t*)(codes + b * 16 + part * 4) = bad ? 0u : c;
            if (part == 0) scales[b] = bad ? 255 : (uint8_t)(X + 127);
        }
    }
}

}  // namespace

hipError_t launch_quant_mxfp4(const void* a, int in_dtype, long long rows, int K, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream) {
    const long long blocks = rows * (K / 32);
    if (blocks == 0) return hipSuccess;
    const long long n = (blocks + 64 * kU - 1) / (64 * kU);
    const unsigned x = (unsigned)(n < (1ll << 20) ? n : 1ll << 20);
    const dim3 grid(x, (unsigned)((n + x - 1) / x));
    if (in_dtype == MOE_IN_F32)
        hipLaunchKernelGGL(quant_mxfp4_kernel<true>, grid, dim3(256), 0, stream, a, codes, scales,
                           blocks);
    else
        hipLaunchKernelGGL(quant_mxfp4_kernel<false>, grid, dim3(256), 0, stream, a, codes, scales,
                           blocks);
    return hipGetLastError();
}

}  // namespace moe
