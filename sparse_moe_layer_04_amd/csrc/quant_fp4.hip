// MXFP4 quantisation of rows: E2M1 codes with one power-of-two scale for each
// 32 values,
//   X = floor(log2(max |v|)) - 2 in [-127, 127] (0 for zeros), scale byte
//   X + 127; code = E2M1(v / 2^X), nearest, ties to even, saturating at +-6;
// a block that holds an infinity or NaN gets the scale byte 255 (NaN).
// v / 2^X is exact (a power of two; where it is subnormal the code is 0 on
// either side of its rounding).
//
// The rows are one run of blocks (K is a multiple of 32), so a thread takes a
// block whatever K is: 64 or 128 bytes in, a 16-byte store of codes out.
#include "fp4.h"

namespace moe {
namespace {

// E2M1 code of m >= 0 (sign apart): the count of the midpoints below m, the
// ties (at 0.25, 1.25 and 2.5 and 5 down, at 0.75, 1.75 and 3.5 up) to even
__device__ __forceinline__ uint32_t e2m1(float v) {
    const float m = fabsf(v);
    const uint32_t c = (m > 0.25f) + (m >= 0.75f) + (m > 1.25f) + (m >= 1.75f) + (m > 2.5f) +
                       (m >= 3.5f) + (m > 5.0f);
    return c | (__float_as_uint(v) >> 31) << 3;
}

template <bool F32>
__global__ __launch_bounds__(256) void quant_mxfp4_kernel(const void* __restrict__ a,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales,
                                                          long long blocks) {
    const long long b = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (b >= blocks) return;
    float v[32];
    const u32x4* src = (const u32x4*)((const uint8_t*)a + (size_t)b * (F32 ? 128 : 64));
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) {
        const u32x4 w = src[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (F32) {
                v[4 * i + j] = __uint_as_float(w[j]);
            } else {
                v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
    uint32_t top = 0;                      // |v| as bits: infinities and NaN are the largest
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    // (a subnormal maximum has exponent field 0: X = -127 as for all below 2^-124)
    int X = top == 0 ? 0 : max((int)(top >> 23) - 129, -127);
    const bool bad = top >= 0x7f800000u;
    const float inv = __uint_as_float((uint32_t)(127 - X) << 23);  // 2^-X: X in [-127, 126]
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) c |= e2m1(v[8 * i + j] * inv) << (4 * j);
        out[i] = bad ? 0u : c;
    }
    *(u32x4*)(codes + b * 16) = out;
    scales[b] = bad ? 255 : (uint8_t)(X + 127);
}

}  // namespace

hipError_t launch_quant_mxfp4(const void* a, int in_dtype, long long rows, int K, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream) {
    const long long blocks = rows * (K / 32);
    if (blocks == 0) return hipSuccess;
    const long long n = (blocks + 255) / 256;
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
