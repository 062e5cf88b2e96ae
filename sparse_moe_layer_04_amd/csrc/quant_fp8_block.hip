// 128-block 8-bit quantisation: E4M3 codes with one power-of-two fp32 scale
// for each block of 128 values of a row (activations, gradients), or for each
// 128 x 128 block of a matrix (weights).
//
//   X = the least integer with max |v| <= 448 * 2^X, in [-126, 120] (0 for a
//       block of zeros), scale = 2^X, code = E4M3(v / 2^X), nearest, ties to
//       even.
// With the least such X the block's largest value lands in (224, 448], so no
// value saturates and v / 2^X is exact.  X from amax = m 2^e, m in [1, 2):
// 448 = 1.75 * 2^8, so X = e - 8 when m <= 1.75 and e - 7 above.
// A value that is not finite takes no part in the maximum and its code is
// E4M3's NaN, so that an overflow stays visible behind the quantiser.
//
// Bound: HBM, each value read once and its code written once (3 bytes a bf16
// value, 5 an fp32 one); a block is held in registers between the maximum
// and the conversion.  Lanes are laid along the row (8 bf16 or 4 fp32 values,
// 16 bytes, a lane; 16 or 32 lanes a block), so every load and store
// instruction of a wave covers whole lines.  8191 x 2000 fp32 values: 15.5 us
// (5.3 TB/s); 39043 x 4080: 154 us (5.2 TB/s); weights of 64 x 1024 x 2048
// bf16: 76.7 us (5.3 TB/s).  64 x 4096 bf16 values: 3.5 us, a launch.
#include "fp8_block.h"

namespace moe {
namespace {

// A launch's x extent holds fewer than 2^32 threads, which are 2^24 workgroups
// of 256: beyond kGridX workgroups there are rows of them.
constexpr unsigned kGridX = 1u << 20;
dim3 grid_of(unsigned n) {
    const unsigned x = n < kGridX ? n : kGridX;
    return dim3(x, (n + x - 1) / x);
}
__device__ __forceinline__ unsigned workgroup() { return blockIdx.y * gridDim.x + blockIdx.x; }

// values of one 16-byte load: 8 bf16 or 4 fp32
template <bool F32>
struct Ld {
    static constexpr int V = F32 ? 4 : 8;       // values a lane
    static constexpr int L = 128 / V;           // lanes a block of 128
};

template <bool F32>
__device__ __forceinline__ float value(const u32x4& w, int i) {
    if constexpr (F32) return __uint_as_float(w[i]);
    const uint32_t u = w[i >> 1];
    return __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
}

template <bool F32>
__device__ __forceinline__ float lane_amax(const u32x4& w) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < Ld<F32>::V; ++i) m = fmaxf(m, finite_abs(value<F32>(w, i)));
    return m;
}

// codes of the lane's values times the exact power of two inv: 8 or 4 bytes
template <bool F32>
__device__ __forceinline__ void lane_codes(const u32x4& w, float inv, uint8_t* dst) {
    uint32_t c[Ld<F32>::V / 4];
#pragma unroll
    for (int i = 0; i < Ld<F32>::V / 4; ++i)
        c[i] = e4m3_pack4(value<F32>(w, 4 * i), value<F32>(w, 4 * i + 1), value<F32>(w, 4 * i + 2),
                          value<F32>(w, 4 * i + 3), inv);
    if constexpr (F32)
        *(uint32_t*)dst = c[0];
    else
        *(u32x2*)dst = u32x2{c[0], c[1]};
}

// Rows: 16 (32) lanes a block; a thread takes kU blocks, their loads in
// flight together.
constexpr int kU = 4;

template <bool F32>
__global__ __launch_bounds__(256) void quant_rows_kernel(const void* __restrict__ a,
                                                         uint8_t* __restrict__ codes,
                                                         float* __restrict__ scales,
                                                         unsigned nblocks, int K, int nb) {
    constexpr int V = Ld<F32>::V, L = Ld<F32>::L, PB = 256 / L;
    const int li = threadIdx.x % L;
    // (past the last block: a workgroup of the last row of them has none)
    const unsigned first = min(workgroup(), (nblocks - 1) / (PB * kU) + 1) * (unsigned)(PB * kU) +
                           threadIdx.x / L;
    u32x4 w[kU];
    size_t at[kU];
    bool live[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const unsigned s = first + u * PB;
        const unsigned row = s / (unsigned)nb, b = s - row * (unsigned)nb;
        const int c = (int)b * 128 + li * V;
        live[u] = s < nblocks && c < K;
        at[u] = (size_t)row * K + c;
        w[u] = u32x4{0u, 0u, 0u, 0u};
        if (live[u]) w[u] = *(const u32x4*)((const uint8_t*)a + at[u] * (F32 ? 4 : 2));
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        float m = row16_max(lane_amax<F32>(w[u]));
        if constexpr (L == 32) m = fmaxf(m, __shfl_xor(m, 16, 64));
        const int X = block_exponent(m);
        if (live[u]) lane_codes<F32>(w[u], pow2(-X), codes + at[u]);
        const unsigned s = first + u * PB;
        if (li == 0 && s < nblocks) scales[s] = pow2(X);
    }
}

// Matrices: one workgroup per 128 x 128 block, its values in registers (8 or
// 16 loads a thread) between the maximum and the conversion.
template <bool F32>
__global__ __launch_bounds__(256) void quant_matrix_kernel(const void* __restrict__ a,
                                                           uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales, int N,
                                                           int K, int nbn, int nbk,
                                                           unsigned nblocks) {
    constexpr int V = Ld<F32>::V, L = Ld<F32>::L, PR = 256 / L, NP = 128 / PR;
    __shared__ float part[4];
    const unsigned blk = workgroup();
    if (blk >= nblocks) return;
    const unsigned kb = blk % (unsigned)nbk, rest = blk / (unsigned)nbk;
    const unsigned rb = rest % (unsigned)nbn, g = rest / (unsigned)nbn;
    const int c = (int)kb * 128 + (threadIdx.x % L) * V;
    const int r0 = (int)rb * 128 + threadIdx.x / L;
    const size_t base = ((size_t)g * N + r0) * K + c;
    u32x4 w[NP];
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        w[p] = u32x4{0u, 0u, 0u, 0u};
        if (c < K && r0 + p * PR < N)
            w[p] = *(const u32x4*)((const uint8_t*)a +
                                   (base + (size_t)(p * PR) * K) * (F32 ? 4 : 2));
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) m = fmaxf(m, lane_amax<F32>(w[p]));
    m = row16_max(m);
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const int X = block_exponent(m);
    const float inv = pow2(-X);
#pragma unroll
    for (int p = 0; p < NP; ++p)
        if (c < K && r0 + p * PR < N)
            lane_codes<F32>(w[p], inv, codes + base + (size_t)(p * PR) * K);
    if (threadIdx.x == 0) scales[blk] = pow2(X);
}

}  // namespace

hipError_t launch_quant_rows_fp8_block(const void* a, int in_dtype, long long rows, int K,
                                       uint8_t* codes, float* scales, hipStream_t stream) {
    const int nb = (int)block_count(K);
    const unsigned nblocks = (unsigned)(rows * nb);
    if (nblocks == 0) return hipSuccess;
    const unsigned per = (in_dtype == MOE_IN_F32 ? 8u : 16u) * kU;
    const dim3 grid = grid_of((nblocks + per - 1) / per);
    if (in_dtype == MOE_IN_F32)
        hipLaunchKernelGGL(quant_rows_kernel<true>, grid, dim3(256), 0, stream, a, codes, scales,
                           nblocks, K, nb);
    else
        hipLaunchKernelGGL(quant_rows_kernel<false>, grid, dim3(256), 0, stream, a, codes, scales,
                           nblocks, K, nb);
    return hipGetLastError();
}

hipError_t launch_quant_matrix_fp8_block(const void* w, int in_dtype, int G, int N, int K,
                                         uint8_t* codes, float* scales, hipStream_t stream) {
    const int nbn = (int)block_count(N), nbk = (int)block_count(K);
    const unsigned nblocks = (unsigned)((long long)G * nbn * nbk);
    const dim3 grid = grid_of(nblocks);
    if (in_dtype == MOE_IN_F32)
        hipLaunchKernelGGL(quant_matrix_kernel<true>, grid, dim3(256), 0, stream, w, codes, scales,
                           N, K, nbn, nbk, nblocks);
    else
        hipLaunchKernelGGL(quant_matrix_kernel<false>, grid, dim3(256), 0, stream, w, codes,
                           scales, N, K, nbn, nbk, nblocks);
    return hipGetLastError();
}

}  // namespace moe
