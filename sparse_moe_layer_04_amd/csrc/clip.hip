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
// ones first: what the first pass read last is still in the cache.  A chunk's
// loads are issued a chunk ahead and its address two ahead.  The second pass
// loads and stores past the caches (nontemporal): 409 M fp32 values 888 us ->
// 831, 40 M 80 -> 75; the first pass too 804, but 83 and, with 100 M, 190 ->
// 201 (what it leaves in the cache is then lost).
//
// Bound: HBM, 12 bytes an fp32 value (the second read is real where the
// gradients pass the cache's 256 MB): 409 M values 815 us, 6.0 TB/s, the rate
// of a large copy; 100 M 181 us; 40 M 79 (6.1).  400 tensors of 3 M values in
// all 11.6 us, two launches of 3 and 6 and the host's call; with loops over a
// short chunk's pieces and the norm added before the first values were asked
// for 14.0.  In place 409 M values take 823 us, within the limit 500 (the norm
// alone 268): there the second pass writes nothing, but its loads are on their way
// before the norm is known.
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

constexpr int kU = kGradChunk / 4 / kT;    // 16-byte pieces a thread, of an fp32 chunk

// A chunk's values on their way: pieces threadIdx.x + 256 u, the last one again
// beyond it, and of the values behind the pieces one a thread.  (In a loop over
// the pieces of short chunks each load would wait for the one before.)
// ONCE: they are not read again soon.
template <bool ONCE>
struct Load {
    GradChunk c;
    u32x4 w[kU];
    uint32_t value;                        // the one behind the pieces
    int pieces, rest;                      // whole ones of 16 bytes; the value's place

    __device__ __forceinline__ void issue(const GradChunk& chunk) {
        c = chunk;
        pieces = c.n / (c.f32 ? 4 : 8);
        const int inside = pieces * (c.f32 ? 4 : 8);
        rest = inside + (int)threadIdx.x;
        const u32x4* g = (const u32x4*)c.grad;
        auto load = [&](int u) {
            const u32x4* at = g + min(u * kT + (int)threadIdx.x, pieces - 1);
            w[u] = ONCE ? __builtin_nontemporal_load(at) : *at;
        };
        if (pieces > 0)
#pragma unroll
            for (int u = 0; u < kU / 2; ++u) load(u);
        if (pieces > kU / 2 * kT)
#pragma unroll
            for (int u = kU / 2; u < kU; ++u) load(u);
        if (inside < c.n && rest < c.n)
            value = c.f32 ? ((const uint32_t*)c.grad)[rest]
                          : (uint32_t)((const uint16_t*)c.grad)[rest] << 16;
    }
    // f(u, place) for this thread's pieces
    template <class F>
    __device__ __forceinline__ void each(const F& f) const {
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (u * kT + (int)threadIdx.x < pieces) f(u, u * kT + (int)threadIdx.x);
    }
};

__global__ __launch_bounds__(kT) void grad_square_kernel(const GradChunk* __restrict__ plan,
                                                         long long chunks,
                                                         double* __restrict__ part) {
    double sum = 0.0;
    long long at = blockIdx.x;
    Load<false> next;
    next.issue(plan[at]);
    GradChunk after = plan[at + gridDim.x < chunks ? at + gridDim.x : at];
    while (at < chunks) {
        const Load<false> l = next;
        at += gridDim.x;
        if (at < chunks) {
            next.issue(after);
            after = plan[at + gridDim.x < chunks ? at + gridDim.x : at];
        }
        if (l.c.f32) l.each([&](int u, int) { sum += square_sum(l.w[u], true); });
        else l.each([&](int u, int) { sum += square_sum(l.w[u], false); });
        if (l.rest < l.c.n) {
            const double v = __uint_as_float(l.value);
            sum = __builtin_fma(v, v, sum);
        }
    }
    sum = group_sum(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// the norm from the partial sums, in every thread
__device__ __forceinline__ double norm_of(const double* part, int parts) {
    constexpr int kN = kGradParts / kT;
    double p[kN], v = 0.0;
    if (parts > 0)
#pragma unroll
        for (int i = 0; i < kN; ++i) p[i] = part[min(i * kT + (int)threadIdx.x, parts - 1)];
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (i * kT + (int)threadIdx.x < parts) v += p[i];
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
    // (the first chunk's values are on their way while the sums are added)
    long long at = chunks - 1 - blockIdx.x;
    auto plan_at = [&](long long i) { return plan[i >= 0 ? i : 0]; };
    Load<true> next;
    GradChunk after;
    if (chunks > 0) {
        next.issue(plan_at(at));
        after = plan_at(at - gridDim.x);
    }
    const double total = norm_of(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
    const bool clip = total > max_norm && total < __builtin_inf();
    const double f = clip ? max_norm / total : 1.0;
    // (in place and within the norm there is nothing to write)
    while (at >= 0) {
        const Load<true> l = next;
        at -= gridDim.x;
        if (at >= 0) {
            next.issue(after);
            after = plan_at(at - gridDim.x);
        }
        if (!clip && l.c.out == l.c.grad) continue;
        u32x4* o = (u32x4*)l.c.out;
        auto store = [&](bool f32) {
            l.each([&](int u, int i) {
                __builtin_nontemporal_store(clip ? scaled16(l.w[u], f32, f) : l.w[u], o + i);
            });
        };
        if (l.c.f32) store(true);
        else store(false);
        if (l.rest < l.c.n) {
            const float v = clip ? scaled(__uint_as_float(l.value), f) : __uint_as_float(l.value);
            if (l.c.f32) ((float*)l.c.out)[l.rest] = v;
            else ((uint16_t*)l.c.out)[l.rest] =
                (uint16_t)(clip ? bf16_pack2(v, 0.0f) : l.value >> 16);
        }
    }
}

int parts_of(long long chunks) { return (int)(chunks < kGradParts ? chunks : kGradParts); }
// more workgroups than are resident scale 1 to 2% faster (409 M values: 831 us
// with 2048, 827 with 4096, 820 with 8192)
int scalers_of(long long chunks) { return (int)(chunks < 8192 ? chunks : 8192); }

}  // namespace

hipError_t launch_grad_norm(const GradChunk* plan, long long chunks, double* part, float* norm,
                            hipStream_t stream) {
    const int parts = parts_of(chunks);
    if (parts > 0)
        hipLaunchKernelGGL(grad_square_kernel, dim3(parts), dim3(kT), 0, stream, plan, chunks,
                           part);
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kT), 0, stream, part, parts, norm);
    return hipGetLastError();
}

hipError_t launch_clip_grad_norm(const GradChunk* plan, long long chunks, double max_norm,
                                 double* part, float* norm, hipStream_t stream) {
    const int parts = parts_of(chunks);
    if (parts > 0)
        hipLaunchKernelGGL(grad_square_kernel, dim3(parts), dim3(kT), 0, stream, plan, chunks,
                           part);
    hipLaunchKernelGGL(grad_scale_kernel, dim3(parts > 0 ? scalers_of(chunks) : 1), dim3(kT), 0,
                       stream, plan, chunks, max_norm, part, parts, norm);
    return hipGetLastError();
}

}  // namespace moe
