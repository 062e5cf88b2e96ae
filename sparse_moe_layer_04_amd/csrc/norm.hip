// Root-mean-square norm with the residual's addition, and its backward.
//
//   s = x + residual, rounded to the residual's type,
//   n = fl32(s / sqrt(mean(s^2) + eps)), y = fl32(n w),
// y to bf16, and to E4M3 codes with a power-of-two scale for each 128 values
// (the rule of moe_quantize_fp8_block, on the fp32 y).  The sum of squares,
// the root and s / root are held in 64 bits: no sum overflows or vanishes
// (|s| up to the type's largest), and y comes out the same bits for any order
// of the sum, so that codes and scales next to a border do too.
#include "step.h"

namespace moe {
namespace {

// A launch's x extent holds fewer than 2^32 threads: beyond kGridX workgroups
// there are rows of them.
constexpr unsigned kGridX = 1u << 20;
dim3 grid_of(long long n) {
    const unsigned x = (unsigned)(n < (long long)kGridX ? n : (long long)kGridX);
    return dim3(x, (unsigned)((n + x - 1) / x));
}
__device__ __forceinline__ long long workgroup() {
    return (long long)blockIdx.y * gridDim.x + blockIdx.x;
}

// W waves a row (blockDim.x / 64 of them, or 1 with a row for every wave of
// the workgroup), NC chunks of 8 values a lane: chunk c of lane l of the row's
// wave w holds values 8 (64 (W c + w) + l) + (0 .. 7), so 16 lanes hold a
// block of 128.
template <int NC, bool ONE>
__global__ __launch_bounds__(ONE ? 256 : 1024) void add_rms_norm_kernel(NormArgs p) {
    __shared__ double part[ONE ? 1 : 16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int W = ONE ? 1 : (int)(blockDim.x >> 6), d = p.d;
    const long long row = ONE ? workgroup() * 4 + wave : workgroup();
    if (row >= p.rows) return;
    const size_t at = (size_t)row * d;
    const int first = 8 * ((ONE ? 0 : wave * 64) + lane), step = 512 * W;
    float s[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first + c * step;
#pragma unroll
        for (int j = 0; j < 8; ++j) s[c][j] = 0.0f;
        if (i < d) load8(p.x, at + i, p.x_f32, s[c]);
    }
    if (p.res) {
        float r[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (first + c * step < d) load8(p.res, at + first + c * step, p.res_f32, r[c]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first + c * step;
            if (i >= d) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) s[c][j] += r[c][j];
            if (!p.res_f32) {
                const u32x4 b = bf16_pack8(s[c]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[c][2 * j] = __uint_as_float(b[j] << 16);
                    s[c][2 * j + 1] = __uint_as_float(b[j] & 0xffff0000u);
                }
                *(u32x4*)((uint16_t*)p.res_out + at + i) = b;
            } else {
                store8(p.res_out, at + i, true, s[c]);
            }
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)s[c][j], (double)s[c][j], sum);
    sum = wave_sum(sum);
    if constexpr (!ONE) {
        if (lane == 0) part[wave] = sum;
        __syncthreads();
        sum = part[0];
        for (int w = 1; w < W; ++w) sum += part[w];
    }
    const double rstd = 1.0 / __builtin_sqrt(sum / d + p.eps);
    const int nb = (d + 127) / 128;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int i = first + c * step;
        const bool in = i < d;
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0.0f;
        if (in) load8(p.w, i, p.w_f32, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= (float)((double)s[c][j] * rstd);
        if (in && p.y) store8(p.y, at + i, false, w);
        if (p.codes) {
            float m = 0.0f;
            if (in)
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(w[j]));
            const int X = block_exponent(row16_max(m));
            const float inv = pow2(-X);
            if (in) {
                *(u32x2*)(p.codes + at + i) = u32x2{e4m3_pack4(w[0], w[1], w[2], w[3], inv),
                                                    e4m3_pack4(w[4], w[5], w[6], w[7], inv)};
                if ((lane & 15) == 0) p.scales[(size_t)row * nb + i / 128] = pow2(X);
            }
        }
    }
}

// Backward.  With g = dy w, r = 1 / sqrt(mean(s^2) + eps) and n = s r,
//   dx = r (g - n mean(g n)) + d_res = r g - (r^3 / d) (sum g s) s + d_res,
//   dw = sum_t dy n.
// One pass over a row: the sums of s^2 and of g s together (64 bits, as is the
// last line, whose terms cancel), the row held in registers.  A wave or a
// workgroup takes rows t, t + stride, ... and keeps its columns' dw in
// registers (fp32, at most a few dozen terms each); its sums go to a row of
// `part`, which the second kernel adds up (64 bits), always in the same order.
template <int NC, bool ONE>
__global__ __launch_bounds__(ONE ? 256 : 1024) void rms_norm_backward_kernel(NormBwdArgs p) {
    __shared__ double part[2][ONE ? 1 : 16][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int W = ONE ? 1 : (int)(blockDim.x >> 6), d = p.d;
    const long long slot = ONE ? (long long)blockIdx.x * 4 + wave : (long long)blockIdx.x;
    const long long stride = ONE ? (long long)gridDim.x * 4 : (long long)gridDim.x;
    const int first = 8 * ((ONE ? 0 : wave * 64) + lane), step = 512 * W;
    float dw[NC][8], w[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[c][j] = 0.0f, w[c][j] = 0.0f;
        if (first + c * step < d) load8(p.w, first + c * step, p.w_f32, w[c]);
    }
    int turn = 0;
    for (long long row = slot; row < p.rows; row += stride, turn ^= 1) {
        const size_t at = (size_t)row * d;
        float s[NC][8], dy[NC][8], r[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first + c * step;
#pragma unroll
            for (int j = 0; j < 8; ++j) s[c][j] = 0.0f, dy[c][j] = 0.0f, r[c][j] = 0.0f;
            if (i < d) {
                load8(p.s, at + i, p.s_f32, s[c]);
                load8(p.dy, at + i, p.dy_f32, dy[c]);
                if (p.d_res) load8(p.d_res, at + i, p.res_f32, r[c]);
            }
        }
        double ss = 0.0, gs = 0.0;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double v = s[c][j];
                ss = __builtin_fma(v, v, ss);
                gs = __builtin_fma((double)dy[c][j] * (double)w[c][j], v, gs);
            }
        ss = wave_sum(ss);
        gs = wave_sum(gs);
        if constexpr (!ONE) {
            // (two sets, so that one barrier a row is enough)
            if (lane == 0) part[turn][wave][0] = ss, part[turn][wave][1] = gs;
            __syncthreads();
            ss = part[turn][0][0];
            gs = part[turn][0][1];
            for (int v = 1; v < W; ++v) ss += part[turn][v][0], gs += part[turn][v][1];
        }
        const double rstd = 1.0 / __builtin_sqrt(ss / d + p.eps);
        const double along = gs / d * rstd * rstd * rstd;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i = first + c * step;
            float out[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double g = (double)dy[c][j] * (double)w[c][j];
                out[j] = (float)__builtin_fma(g, rstd,
                                              __builtin_fma(-along, (double)s[c][j],
                                                            (double)r[c][j]));
                dw[c][j] = __builtin_fmaf(dy[c][j], (float)((double)s[c][j] * rstd), dw[c][j]);
            }
            if (i < d) store8(p.dx, at + i, p.dx_f32, out);
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (first + c * step < d)
            store8(p.part, (size_t)slot * d + first + c * step, true, dw[c]);
}

// dw[c] = sum of part[., c]: 32 columns a workgroup, its 32 groups of 8 lanes
// take rows 32 apart
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* __restrict__ part, int parts,
                                                      int d, float* __restrict__ dw) {
    __shared__ double sum[32][33];
    const int li = threadIdx.x & 7, r0 = threadIdx.x >> 3, c = blockIdx.x * 32 + li * 4;
    double a[4] = {0.0, 0.0, 0.0, 0.0};
    if (c < d)
        for (int r = r0; r < parts; r += 32) {
            const f32x4 v = *(const f32x4*)(part + (size_t)r * d + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] += (double)v[j];
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[r0][li * 4 + j] = a[j];
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < d) {
        double v = 0.0;
        for (int r = 0; r < 32; ++r) v += sum[r][threadIdx.x];
        dw[blockIdx.x * 32 + threadIdx.x] = (float)v;
    }
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& p, hipStream_t stream) {
    if (p.rows == 0) return hipSuccess;
    const int chunks = (p.d + 511) / 512;          // of a wave
    const bool many = p.rows >= 1024 && chunks <= 8;
    if (many || chunks == 1) {
        const dim3 grid = grid_of((p.rows + 3) / 4);
        if (chunks <= 1) hipLaunchKernelGGL((add_rms_norm_kernel<1, true>), grid, dim3(256), 0, stream, p);
        else if (chunks <= 2) hipLaunchKernelGGL((add_rms_norm_kernel<2, true>), grid, dim3(256), 0, stream, p);
        else if (chunks <= 4) hipLaunchKernelGGL((add_rms_norm_kernel<4, true>), grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL((add_rms_norm_kernel<8, true>), grid, dim3(256), 0, stream, p);
    } else {
        const dim3 grid = grid_of(p.rows);
        if (chunks <= 16) hipLaunchKernelGGL((add_rms_norm_kernel<1, false>), grid, dim3(64 * chunks), 0, stream, p);
        else if (chunks <= 32) hipLaunchKernelGGL((add_rms_norm_kernel<2, false>), grid, dim3(64 * ((chunks + 1) / 2)), 0, stream, p);
        else hipLaunchKernelGGL((add_rms_norm_kernel<4, false>), grid, dim3(64 * ((chunks + 3) / 4)), 0, stream, p);
    }
    return hipGetLastError();
}

namespace {
constexpr int kNormParts = 1024;       // rows of `part`, at most
struct NormBwdShape {
    bool one;                          // a wave a row
    int threads, chunks;               // chunks a lane
    int parts;
};
NormBwdShape norm_bwd_shape(long long rows, int d) {
    const int waves = (d + 511) / 512;
    NormBwdShape s;
    s.one = waves <= 2;
    s.chunks = s.one ? waves : waves <= 16 ? 1 : waves <= 32 ? 2 : 4;
    if (!s.one && waves > 4 && waves <= 16) s.chunks = 2;
    s.threads = s.one ? 256 : 64 * ((waves + s.chunks - 1) / s.chunks);
    const long long most = s.one ? (rows + 3) / 4 * 4 : rows;
    s.parts = (int)(most < kNormParts ? most : kNormParts);
    return s;
}
}  // namespace

int norm_backward_parts(long long rows, int d) { return norm_bwd_shape(rows, d).parts; }

hipError_t launch_rms_norm_backward(const NormBwdArgs& p, hipStream_t stream) {
    const NormBwdShape s = norm_bwd_shape(p.rows, p.d);
    if (s.parts > 0) {
        const dim3 grid((unsigned)(s.one ? s.parts / 4 : s.parts)), block(s.threads);
        if (s.one) {
            if (s.chunks == 1) hipLaunchKernelGGL((rms_norm_backward_kernel<1, true>), grid, block, 0, stream, p);
            else hipLaunchKernelGGL((rms_norm_backward_kernel<2, true>), grid, block, 0, stream, p);
        } else if (s.chunks == 1) {
            hipLaunchKernelGGL((rms_norm_backward_kernel<1, false>), grid, block, 0, stream, p);
        } else if (s.chunks == 2) {
            hipLaunchKernelGGL((rms_norm_backward_kernel<2, false>), grid, block, 0, stream, p);
        } else {
            hipLaunchKernelGGL((rms_norm_backward_kernel<4, false>), grid, block, 0, stream, p);
        }
    }
    hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((p.d + 31) / 32)), dim3(256), 0, stream,
                       p.part, s.parts, p.d, p.dw);
    return hipGetLastError();
}

}  // namespace moe
