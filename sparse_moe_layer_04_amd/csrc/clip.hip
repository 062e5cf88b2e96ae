// The norm of many gradient tensors, and their clipping.
//
//   norm = sqrt(sum of all squares), out = g * min(1, max_norm / norm),
// the squares added in 64 bits (no overflow or loss of small ones, and the
// same bits for any split to within 1e-16).  Where the norm is not finite the
// gradients are left as they are (copied to out).
//
// The tensors come as a plan of chunks of 8192 values (address, count, type:
// 32 bytes a chunk, 0.1% of the bytes), so that any number of tensors of any
// sizes is one launch, and a workgroup's next address is one load.
//
// Two launches: partial sums, a workgroup each; then every workgroup adds the
// partial sums (16 KB at most, in the same order) and scales its chunks, last
// ones first: what the first pass read last is still in the cache.
#include "step.h"

namespace moe {
namespace {

constexpr int kT = 256;

// sum of v over the workgroup, in a fixed order, in every thread
__device__ __forceinline__ double group_sum(double v) {
    __shared__ double part[kT / 64];
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) v += part[w];
    return v;
}

__device__ __forceinline__ double square_sum(const u32x4& w, bool f32) {
    double a = 0.0, b = 0.0;
    if (f32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double v = __uint_as_float(w[i]);
            a = __builtin_fma(v, v, a);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double v = __uint_as_float(w[i] << 16), u = __uint_as_float(w[i] & 0xffff0000u);
            a = __builtin_fma(v, v, a);
            b = __builtin_fma(u, u, b);
        }
    }
    return a + b;
}

__device__ __forceinline__ float one_value(const GradChunk& c, int i) {
    return c.f32 ? ((const float*)c.grad)[i] : bf16_to_f32(((const uint16_t*)c.grad)[i]);
}

__global__ __launch_bounds__(kT) void grad_square_kernel(const GradChunk* __restrict__ plan,
                                                         long long chunks,
                                                         double* __restrict__ part) {
    double sum = 0.0;
    for (long long at = blockIdx.x; at < chunks; at += gridDim.x) {
        const GradChunk c = plan[at];
        const int per = c.f32 ? 4 : 8, n = c.n / per;   // 16-byte pieces
        const u32x4* g = (const u32x4*)c.grad;
        constexpr int U = kGradChunk / 4 / kT;
        if (c.n == kGradChunk) {
            u32x4 w[U];
            if (c.f32) {
#pragma unroll
                for (int u = 0; u < U; ++u) w[u] = g[u * kT + threadIdx.x];
#pragma unroll
                for (int u = 0; u < U; ++u) sum += square_sum(w[u], true);
            } else {
#pragma unroll
                for (int u = 0; u < U / 2; ++u) w[u] = g[u * kT + threadIdx.x];
#pragma unroll
                for (int u = 0; u < U / 2; ++u) sum += square_sum(w[u], false);
            }
        } else {
            for (int i = threadIdx.x; i < n; i += kT) sum += square_sum(g[i], c.f32);
            const int rest = n * per + (int)threadIdx.x;
            if (rest < c.n) {
                const double v = one_value(c, rest);
                sum = __builtin_fma(v, v, sum);
            }
        }
    }
    sum = group_sum(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// the norm from the partial sums, in every thread
__device__ __forceinline__ double norm_of(const double* part, int parts) {
    double v = 0.0;
    for (int i = threadIdx.x; i < parts; i += kT) v += part[i];
    return __builtin_sqrt(group_sum(v));
}

__global__ __launch_bounds__(kT) void grad_norm_kernel(const double* __restrict__ part, int parts,
                                                       float* __restrict__ norm) {
    const double n = norm_of(part, parts);
    if (threadIdx.x == 0) *norm = (float)n;
}

__device__ __forceinline__ float scaled(float v, double f) { return (float)((double)v * f); }

__device__ __forceinline__ u32x4 scaled16(const u32x4& w, bool f32, double f) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = f32 ? __float_as_uint(scaled(__uint_as_float(w[i]), f))
                   : bf16_pack2(scaled(__uint_as_float(w[i] << 16), f),
                                scaled(__uint_as_float(w[i] & 0xffff0000u), f));
    return r;
}

__global__ __launch_bounds__(kT) void grad_scale_kernel(const GradChunk* __restrict__ plan,
                                                        long long chunks, double max_norm,
                                                        const double* __restrict__ part, int parts,
                                                        float* __restrict__ norm) {
    const double total = norm_of(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
    const bool clip = total > max_norm && total < __builtin_inf();
    const double f = clip ? max_norm / total : 1.0;
    for (long long at = chunks - 1 - blockIdx.x; at >= 0; at -= gridDim.x) {
        const GradChunk c = plan[at];
        if (!clip && c.out == c.grad) continue;
        const int per = c.f32 ? 4 : 8, n = c.n / per;
        const u32x4* g = (const u32x4*)c.grad;
        u32x4* o = (u32x4*)c.out;
        constexpr int U = kGradChunk / 4 / kT;
        if (c.n == kGradChunk) {
            u32x4 w[U];
            if (c.f32) {
#pragma unroll
                for (int u = 0; u < U; ++u) w[u] = g[u * kT + threadIdx.x];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    o[u * kT + threadIdx.x] = clip ? scaled16(w[u], true, f) : w[u];
            } else {
#pragma unroll
                for (int u = 0; u < U / 2; ++u) w[u] = g[u * kT + threadIdx.x];
#pragma unroll
                for (int u = 0; u < U / 2; ++u)
                    o[u * kT + threadIdx.x] = clip ? scaled16(w[u], false, f) : w[u];
            }
        } else {
            for (int i = threadIdx.x; i < n; i += kT)
                o[i] = clip ? scaled16(g[i], c.f32, f) : g[i];
            const int rest = n * per + (int)threadIdx.x;
            if (rest < c.n) {
                if (c.f32) {
                    const float v = ((const float*)c.grad)[rest];
                    ((float*)c.out)[rest] = clip ? scaled(v, f) : v;
                } else {
                    const uint16_t v = ((const uint16_t*)c.grad)[rest];
                    ((uint16_t*)c.out)[rest] =
                        clip ? (uint16_t)bf16_pack2(scaled(bf16_to_f32(v), f), 0.0f) : v;
                }
            }
        }
    }
}

int parts_of(long long chunks) { return (int)(chunks < kGradParts ? chunks : kGradParts); }

}  // namespace

hipError_t launch_grad_norm(const GradChunk* plan, long long chunks, double* part, float* norm,
                            hipStream_t stream) {
    const int parts = parts_of(chunks);
    if (parts > 0)
        hipLaunchKernelGGL(grad_square_kernel, dim3(parts), dim3(kT), 0, stream, plan, chunks, part);
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kT), 0, stream, part, parts, norm);
    return hipGetLastError();
}

hipError_t launch_clip_grad_norm(const GradChunk* plan, long long chunks, double max_norm,
                                 double* part, float* norm, hipStream_t stream) {
    const int parts = parts_of(chunks);
    if (parts > 0)
        hipLaunchKernelGGL(grad_square_kernel, dim3(parts), dim3(kT), 0, stream, plan, chunks, part);
    hipLaunchKernelGGL(grad_scale_kernel, dim3(parts > 0 ? parts : 1), dim3(kT), 0, stream, plan,
                       chunks, max_norm, part, parts, norm);
    return hipGetLastError();
}

}  // namespace moe
