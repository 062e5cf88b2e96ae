// Root-mean-square norm with the residual's addition, and its backward.
//
//   s = x + residual, rounded to the residual's type,
//   n = fl32(s / sqrt(mean(s^2) + eps)), y = fl32(n w),
// y to bf16, and to E4M3 codes with a power-of-two scale for each 128 values
// (the rule of moe_quantize_fp8_block, on the fp32 y).  The sum of squares,
// the root and s / root are held in 64 bits: no sum overflows or vanishes
// (|s| up to the type's largest), and n depends on the order of the sum only
// where s / root lies within 2^-52 of a border of fp32 (one value in 2^28), so
// that codes and scales next to a border do not either.
//
// Bound: HBM, each value read and written once, 9 bytes a value with a bf16
// residual, bf16 and 8-bit output: 8192 x 4096 54.6 us, 5.6 TB/s (a large copy:
// 6.0); without the residual and the codes, 8191 x 4096, 21.8 us (6.2, half of
// it from the cache).  Loads behind a branch on the type, which the compiler
// waits for one by one, took 93 us: types are template arguments.  Stores or
// loads past the caches: none or slower.  Four rows of 2048: 2.7 us, a launch.
#include <algorithm>
#include <type_traits>

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

// eight weights at i
__device__ __forceinline__ void load_w(const void* w, bool f32, int i, float (&v)[8]) {
    if (f32) {
        Raw8<true> r;
        r.load(w, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r.get(j);
    } else {
        Raw8<false> r;
        r.load(w, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r.get(j);
    }
}

enum Res : int { RES_NONE = 0, RES_BF16 = 1, RES_F32 = 2 };

// W waves a row (those of the workgroup; or ONE, a row for every wave), NC
// chunks of 8 values a lane: chunk c of lane l of the row's wave w holds values
// 8 (64 (W c + w) + l) + (0 .. 7), so 16 lanes hold a block of 128.  (Lanes
// past d load the row's start, so that no load stands behind a branch.)
template <bool XF32, int RES, int NC, bool ONE>
__global__ __launch_bounds__(ONE ? 256 : 1024) void add_rms_norm_kernel(NormArgs p) {
    __shared__ double part[ONE ? 1 : 16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int W = ONE ? 1 : (int)(blockDim.x >> 6), d = p.d, nb = (d + 127) / 128;
    const long long row = ONE ? workgroup() * 4 + wave : workgroup();
    if (row >= p.rows) return;
    const int first = 8 * ((ONE ? 0 : wave * 64) + lane), step = 512 * W;
    int at[NC];
    bool in[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        in[c] = first + c * step < d;
        at[c] = in[c] ? first + c * step : 0;
    }
    Raw8<XF32> x[NC];
    Raw8<RES == RES_F32> r[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) x[c].load(p.x, (size_t)row * d + at[c]);
    if constexpr (RES != RES_NONE)
#pragma unroll
        for (int c = 0; c < NC; ++c) r[c].load(p.res, (size_t)row * d + at[c]);
    float w[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) load_w(p.w, p.w_f32, at[c], w[c]);
    float s[NC][8];
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[c][j] = x[c].get(j);
            if constexpr (RES != RES_NONE) s[c][j] += r[c].get(j);
        }
        const size_t to = (size_t)row * d + at[c];
        if constexpr (RES == RES_BF16) {
            Raw8<false> b;
            b.v[0] = bf16_pack8(s[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[c][j] = b.get(j);
            if (in[c]) *(u32x4*)((uint16_t*)p.res_out + to) = b.v[0];
        }
        if constexpr (RES == RES_F32)
            if (in[c]) store8(p.res_out, to, true, s[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double v = in[c] ? (double)s[c][j] : 0.0;
            sum = __builtin_fma(v, v, sum);
        }
    }
    sum = wave_sum(sum);
    if constexpr (!ONE) {
        if (lane == 0) part[wave] = sum;
        __syncthreads();
        sum = part[0];
        for (int v = 1; v < W; ++v) sum += part[v];
    }
    const double rstd = 1.0 / __builtin_sqrt(sum / d + p.eps);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const size_t to = (size_t)row * d + at[c];
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = w[c][j] * (float)((double)s[c][j] * rstd);
        if (p.y && in[c]) store8(p.y, to, false, y);
        if (p.codes) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(y[j]));
            const int X = block_exponent(row16_max(in[c] ? m : 0.0f));
            const float inv = pow2(-X);
            if (in[c]) {
                *(u32x2*)(p.codes + to) = u32x2{e4m3_pack4(y[0], y[1], y[2], y[3], inv),
                                                e4m3_pack4(y[4], y[5], y[6], y[7], inv)};
                if ((lane & 15) == 0) p.scales[(size_t)row * nb + at[c] / 128] = pow2(X);
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
// registers (fp32); its sums go to a row of `part`, which the second kernel
// adds up (64 bits), always in the same order.  A launch gives each at most
// kNormRun rows, so that no fp32 sum is longer (16384 equal terms were off by
// 2^-12): one launch up to 262144 rows, 524288 of up to 2048 values.  (Runs in a
// loop of the kernel's own cost registers: 8191 x 4104 bf16 73 -> 79 us.)
//
// Bound: HBM, 14 bytes a value with fp32 gradients: 8192 x 4096 84 us + 4.5 for
// the sums of dw, 5.3 TB/s over both.  The last line in 32 bits: the same time.
// AHEAD: the next row's loads before this row's sums, where two rows of bf16
// gradients fit the registers: 8191 x 4096 58 us instead of 63, 16383 x 512 21
// instead of 23; with fp32 ones, spilled, 93 instead of 90.
// Two chunks a lane (rows past 8192): the values are converted to 64 bits a
// second time, not kept so in registers that there are not: 2047 x 16384 bf16
// 75 us instead of 127 (with one chunk, where they fit, 68 instead of 63).
template <bool SF32, bool GF32, int RES, int NC, bool ONE>
__global__ __launch_bounds__(ONE ? 256 : 1024) void rms_norm_backward_kernel(NormBwdArgs p) {
    __shared__ double part[2][ONE ? 1 : 16][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int W = ONE ? 1 : (int)(blockDim.x >> 6), d = p.d;
    const long long slot = ONE ? (long long)blockIdx.x * 4 + wave : (long long)blockIdx.x;
    const long long stride = ONE ? (long long)gridDim.x * 4 : (long long)gridDim.x;
    const int first = 8 * ((ONE ? 0 : wave * 64) + lane), step = 512 * W;
    int at[NC];
    bool in[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        in[c] = first + c * step < d;
        at[c] = in[c] ? first + c * step : 0;
    }
    constexpr bool AHEAD = NC == 1 && !GF32 && RES != RES_F32;
    Raw8<SF32> s[NC], s1[NC];
    Raw8<GF32> g[NC], g1[NC];
    Raw8<RES == RES_F32> r[NC], r1[NC];
    auto load = [&](long long t) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            s1[c].load(p.s, (size_t)t * d + at[c]);
            g1[c].load(p.dy, (size_t)t * d + at[c]);
            if constexpr (RES != RES_NONE) r1[c].load(p.d_res, (size_t)t * d + at[c]);
        }
    };
    if (slot < p.rows) load(slot);
    float dw[NC][8], w[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        load_w(p.w, p.w_f32, at[c], w[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[c][j] = 0.0f;
            w[c][j] = in[c] ? w[c][j] : 0.0f;
        }
    }
    int turn = 0;
    for (long long row = slot; row < p.rows; row += stride, turn ^= 1) {
        double ss = 0.0, gs = 0.0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            s[c] = s1[c];
            g[c] = g1[c];
            // (lanes past d add nothing, whatever the row's start holds)
#pragma unroll
            for (int i = 0; i < (GF32 ? 2 : 1); ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) g[c].v[i][j] = in[c] ? g[c].v[i][j] : 0u;
            if constexpr (RES != RES_NONE) r[c] = r1[c];
        }
        if (AHEAD && row + stride < p.rows) load(row + stride);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double v = in[c] ? (double)s[c].get(j) : 0.0;
                ss = __builtin_fma(v, v, ss);
                gs = __builtin_fma((double)g[c].get(j) * (double)w[c][j], v, gs);
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
        if constexpr (NC > 1) {                  // (converted again from here on)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int i = 0; i < (SF32 ? 2 : 1); ++i) asm volatile("" : "+v"(s[c].v[i]));
#pragma unroll
                for (int i = 0; i < (GF32 ? 2 : 1); ++i) asm volatile("" : "+v"(g[c].v[i]));
#pragma unroll
                for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(w[c][j]));
            }
        }
        const double rstd = 1.0 / __builtin_sqrt(ss / d + p.eps);
        const double along = gs / d * rstd * rstd * rstd;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float out[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float dy = g[c].get(j);
                const double v = s[c].get(j);
                double o = RES == RES_NONE ? 0.0 : (double)r[c].get(j);
                o = __builtin_fma(-along, v, o);
                out[j] = (float)__builtin_fma((double)dy * (double)w[c][j], rstd, o);
                dw[c][j] = __builtin_fmaf(dy, (float)(v * rstd), dw[c][j]);
            }
            if (in[c]) store8(p.dx, (size_t)row * d + at[c], p.dx_f32, out);
        }
        if (!AHEAD && row + stride < p.rows) load(row + stride);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (in[c]) store8(p.part, (size_t)slot * d + at[c], true, dw[c]);
}

// dw[c] = sum of part[., c]: 16 columns a workgroup, its 64 groups of 4 lanes
// take rows 64 apart, eight loads in flight
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* __restrict__ part, int parts,
                                                      int d, float* __restrict__ dw) {
    __shared__ double sum[64][17];
    const int li = threadIdx.x & 3, r0 = threadIdx.x >> 2, c = blockIdx.x * 16 + li * 4;
    const float* from = part + (c < d ? c : 0);
    double a[4] = {0.0, 0.0, 0.0, 0.0};
    for (int r = r0; r < parts; r += 64 * 8) {
        f32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = *(const f32x4*)(from + (size_t)min(r + 64 * u, parts - 1) * d);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] += r + 64 * u < parts ? (double)v[u][j] : 0.0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[r0][li * 4 + j] = a[j];
    __syncthreads();
    // 16 threads a column, then one
    const int col = threadIdx.x & 15, q = threadIdx.x >> 4;
    double v = 0.0;
#pragma unroll
    for (int r = 0; r < 4; ++r) v += sum[4 * q + r][col];
    __syncthreads();
    sum[q][col] = v;
    __syncthreads();
    if (threadIdx.x < 16 && blockIdx.x * 16 + threadIdx.x < d) {
        v = 0.0;
#pragma unroll
        for (int r = 0; r < 16; ++r) v += sum[r][threadIdx.x];
        dw[blockIdx.x * 16 + threadIdx.x] = (float)v;
    }
}

// chunks a lane and waves a row
struct Shape {
    bool one;                          // a wave a row
    int chunks, threads;
};
Shape shape_of(int d, int chunks) {
    const int n = (d + 511) / 512;     // chunks of a row, a wave each
    Shape s;
    s.one = n <= chunks;
    s.chunks = s.one ? n : n <= 16 * chunks ? chunks : 2;
    s.threads = s.one ? 256 : 64 * ((n + s.chunks - 1) / s.chunks);
    return s;
}

template <bool XF32, int RES>
void launch_norm(const NormArgs& p, const Shape& s, dim3 grid, hipStream_t stream) {
#define MOE_NORM(NC, ONE)                                                                      \
    hipLaunchKernelGGL((add_rms_norm_kernel<XF32, RES, NC, ONE>), grid, dim3(s.threads), 0,    \
                       stream, p)
    if (s.one && s.chunks == 1) MOE_NORM(1, true);
    else if (s.one) MOE_NORM(2, true);
    else if (s.chunks == 1) MOE_NORM(1, false);
    else MOE_NORM(2, false);
#undef MOE_NORM
}

template <bool SF32, bool GF32, int RES>
void launch_backward(const NormBwdArgs& p, const Shape& s, dim3 grid, hipStream_t stream) {
#define MOE_NORM(NC, ONE)                                                                      \
    hipLaunchKernelGGL((rms_norm_backward_kernel<SF32, GF32, RES, NC, ONE>), grid,             \
                       dim3(s.threads), 0, stream, p)
    if (s.one && s.chunks == 1) MOE_NORM(1, true);
    else if (s.one) MOE_NORM(2, true);
    else if (s.chunks == 1) MOE_NORM(1, false);
    else MOE_NORM(2, false);
#undef MOE_NORM
}

// Rows of the backward's `part` (of a launch): as many workgroups as are resident at
// once, 8 waves for each of 512.  8192 x 4096, fp32: 92 us with 512, 97 with 1024 (half
// of them wait), 101 with 256; 8191 x 1024 (a wave a row): 28.5 us with 1024
// waves, 38 with 2048 (more partial sums).
constexpr int kNormParts = 512;

constexpr int kNormRun = 512;

Shape backward_shape(int d) { return shape_of(d, 1); }
// rows of `part` of a launch
int backward_slots(long long rows, const Shape& s) {
    const long long most = s.one ? (rows + 3) / 4 * 4 : rows;
    const long long slots = s.one ? 2 * kNormParts : s.threads <= 256 ? 2 * kNormParts : kNormParts;
    return (int)(most < slots ? most : slots);
}
// and of all launches
int backward_parts(long long rows, int slots) {
    const long long each = (long long)slots * kNormRun;
    return slots ? (int)((rows + each - 1) / each * slots) : 0;
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& p, hipStream_t stream) {
    if (p.rows == 0) return hipSuccess;
    // Two loads in flight a lane: of x and the residual, or of two chunks of x
    // (8192 x 4096 bf16: with a residual 54.6 us, with two chunks 58.4; without
    // one 24.4 with one chunk, 21.8 with two).  One chunk where a row's chain of
    // waits is what counts.
    const Shape s = shape_of(p.d, p.rows < 1024 || p.res ? 1 : 2);
    const dim3 grid = grid_of(s.one ? (p.rows + 3) / 4 : p.rows);
    const int res = !p.res ? RES_NONE : p.res_f32 ? RES_F32 : RES_BF16;
    if (p.x_f32) {
        if (res == RES_NONE) launch_norm<true, RES_NONE>(p, s, grid, stream);
        else if (res == RES_BF16) launch_norm<true, RES_BF16>(p, s, grid, stream);
        else launch_norm<true, RES_F32>(p, s, grid, stream);
    } else {
        if (res == RES_NONE) launch_norm<false, RES_NONE>(p, s, grid, stream);
        else if (res == RES_BF16) launch_norm<false, RES_BF16>(p, s, grid, stream);
        else launch_norm<false, RES_F32>(p, s, grid, stream);
    }
    return hipGetLastError();
}

int norm_backward_parts(long long rows, int d) {
    return backward_parts(rows, backward_slots(rows, backward_shape(d)));
}

hipError_t launch_rms_norm_backward(const NormBwdArgs& args, hipStream_t stream) {
    const Shape s = backward_shape(args.d);
    const int slots = backward_slots(args.rows, s), parts = backward_parts(args.rows, slots);
    const long long each = (long long)slots * kNormRun;
    for (long long row = 0; row < args.rows; row += each) {
        NormBwdArgs p = args;
        auto behind = [&](const void* q, int f32) {
            return (const char*)q + (size_t)row * p.d * (f32 ? 4 : 2);
        };
        p.rows = std::min(each, args.rows - row);
        p.s = behind(args.s, p.s_f32);
        p.dy = behind(args.dy, p.dy_f32);
        if (p.d_res) p.d_res = behind(args.d_res, p.res_f32);
        p.dx = const_cast<char*>(behind(args.dx, p.dx_f32));
        p.part = args.part + (size_t)(row / kNormRun) * p.d;
        const dim3 grid((unsigned)(s.one ? slots / 4 : slots));
        const int res = !p.d_res ? RES_NONE : p.res_f32 ? RES_F32 : RES_BF16;
        auto by_res = [&](auto sf, auto gf) {
            constexpr bool S = decltype(sf)::value, G = decltype(gf)::value;
            if (res == RES_NONE) launch_backward<S, G, RES_NONE>(p, s, grid, stream);
            else if (res == RES_BF16) launch_backward<S, G, RES_BF16>(p, s, grid, stream);
            else launch_backward<S, G, RES_F32>(p, s, grid, stream);
        };
        using std::false_type;
        using std::true_type;
        if (p.s_f32 && p.dy_f32) by_res(true_type(), true_type());
        else if (p.s_f32) by_res(true_type(), false_type());
        else if (p.dy_f32) by_res(false_type(), true_type());
        else by_res(false_type(), false_type());
    }
    hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((args.d + 15) / 16)), dim3(256), 0, stream,
                       args.part, parts, args.d, args.dw);
    return hipGetLastError();
}

}  // namespace moe
