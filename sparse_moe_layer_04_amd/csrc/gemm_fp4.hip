// Grouped matrix product of MXFP4 rows and weights on row-major codes: for the
// rows r of group g,
//   out[r, n] = sum_b 2^(Xa[r, b] + Xw[g, n, b]) sum_{k in block b} a[r, k] w[g, n, k],
// b the blocks of 32 of K, codes E2M1, scale bytes X + 127 (255: NaN).
//
// The scaled matrix instructions take both operands as they are: lane l holds
// of row (column) l % 32 the 16 bytes of block 2 s + l / 32 of step s, and that
// block's scale byte.
#include "fp4.h"

namespace moe {
namespace {

template <bool F32>
__global__ __launch_bounds__(256) void gemm_mxfp4_kernel(Fp4GemmArgs p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, l32 = lane & 31;
    auto clamped = [&](int v) { return min(max(v, 0), p.rows); };
    int local = blockIdx.x, g = 0, r0 = 0, n = 0;
    for (;; ++g) {
        if (g == p.G) return;
        r0 = clamped(p.offsets[g]);
        n = max(clamped(p.offsets[g + 1]) - r0, 0);
        const int tiles = (n + 31) >> 5;
        if (local < tiles) break;
        local -= tiles;
    }
    const int row = r0 + 32 * local + l32, end = r0 + n;
    const int n0 = (blockIdx.y * 4 + wave) * 32;
    if (n0 >= p.N) return;
    const int nb = p.K / 32;
    const size_t ar = (size_t)min(row, end - 1), wr = (size_t)g * p.N + min(n0 + l32, p.N - 1);
    const u32x4* ac = (const u32x4*)(p.a + ar * (p.K / 2));
    const u32x4* wc = (const u32x4*)(p.w + wr * (p.K / 2));
    const uint8_t* as = p.as + ar * nb;
    const uint8_t* ws = p.ws + wr * nb;
    f32x16 acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (int b = half; b - half < nb; b += 2) {
        const bool in = b < nb;
        u32x4 x = {0u, 0u, 0u, 0u}, y = x;
        int sx = 127, sy = 127;
        if (in) x = wc[b], y = ac[b], sx = ws[b], sy = as[b];
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0},
            v8i{(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0}, acc, 4, 4, 0, sx, 0, sy);
    }
    if (row >= end) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int col = n0 + 8 * q + 4 * half;
        if (col >= p.N) continue;
        const size_t at = (size_t)row * p.N + col;
        if constexpr (F32)
            *(f32x4*)((float*)p.out + at) =
                f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
        else
            *(u32x2*)((uint16_t*)p.out + at) = u32x2{bf16_pack2(acc[4 * q], acc[4 * q + 1]),
                                                     bf16_pack2(acc[4 * q + 2], acc[4 * q + 3])};
    }
}

}  // namespace

hipError_t launch_grouped_gemm_mxfp4(bool f32, const Fp4GemmArgs& g, hipStream_t stream) {
    const dim3 grid((unsigned)(g.rows / 32 + g.G), (unsigned)((g.N + 127) / 128));
    if (f32) hipLaunchKernelGGL(gemm_mxfp4_kernel<true>, grid, dim3(256), 0, stream, g);
    else hipLaunchKernelGGL(gemm_mxfp4_kernel<false>, grid, dim3(256), 0, stream, g);
    return hipGetLastError();
}

}  // namespace moe
