// Balance loss of the router, with per-expert counts, and its gradient.
//
// A group g is the tokens of one sequence and, with a modality, one class.
// With s = S(logits) (the router's scores), c[g, e] the pairs of the group's
// tokens at expert e, T_g its tokens and f = E c / (k T_g),
//   q_t = sum_e f[g, e] s[t, e] / sum_e s[t, e],  loss[g] = mean of q_t over g,
// the same as sum_e f_e P_e with P_e the mean normalised score, but a sum along
// each token's row: no column sums over tokens, and so no atomics on floats.
// The counts are constants, so with u = d_loss[g] / T_g
//   d logits[t, j] = u (f_j - q_t) s_j (1 - s_j) / sum_e s_e.
//
// Passes: the counts (whole numbers, so that atomics do not depend on their
// order), a pass over the logits for q, a mean of q per group; the gradient is
// one more pass over the logits, which finds q again from the row it holds.
#include "route_device.h"
#include "step.h"

namespace moe {
namespace {

__device__ __forceinline__ float wave_sum_f32(float v) {
#define MOE_STEP(CTRL, RM) v += __uint_as_float(dpp_u32<CTRL, RM>(0u, __float_as_uint(v)));
    MOE_STEP(0xB1, 0xf)    // quad_perm [1,0,3,2]
    MOE_STEP(0x4E, 0xf)    // quad_perm [2,3,0,1]
    MOE_STEP(0x141, 0xf)   // row_half_mirror
    MOE_STEP(0x140, 0xf)   // row_mirror
    MOE_STEP(0x142, 0xa)   // row_bcast:15 into rows 1 and 3
    MOE_STEP(0x143, 0xc)   // row_bcast:31 into rows 2 and 3
#undef MOE_STEP
    return lane_read(v, 63);
}

// offset i, within [0, T]
__device__ __forceinline__ int offset_at(const BalanceArgs& p, int i) {
    return p.offsets ? min(max(p.offsets[i], 0), p.T) : i == 0 ? 0 : p.T;
}

// The sequence of token t: the number of i in [1, S] with offsets[i] <= t; S
// where t lies behind the last one, -1 before the first.  Wave-uniform; a
// wave's lanes look at 64 offsets at once (in halves of what is left where
// there are more).
__device__ __forceinline__ int sequence_of(const BalanceArgs& p, int t, int lane) {
    if (!p.offsets) return 0;
    if (t < offset_at(p, 0)) return -1;
    int lo = 0, n = p.S;                   // the answer is in [lo, lo + n]
    while (n > 64) {
        const int mid = n >> 1;
        if (offset_at(p, lo + mid) <= t) {
            lo += mid;
            n -= mid;
        } else {
            n = mid - 1;
        }
    }
    const bool before = lane < n && offset_at(p, lo + 1 + min(lane, n - 1)) <= t;
    return lo + __popcll(__builtin_amdgcn_ballot_w64(before));
}

// Whether token t's ids are all experts
__device__ __forceinline__ bool ids_valid(const BalanceArgs& p, int t) {
    bool ok = true;
    for (int j = 0; j < p.k; ++j) {
        const int e = p.ids[(size_t)t * p.k + j];
        ok &= e >= 0 && e < p.E;
    }
    return ok;
}

// ---- counts: a workgroup takes kTok tokens.  Where the counts of all the
// sequences among them fit in LDS they are made there and added to the whole
// once a workgroup (an expert's count takes one atomic for many pairs).
constexpr int kTok = 1024;
constexpr int kHist = 15360;               // LDS counters: 60 KB

__global__ __launch_bounds__(256) void balance_zero_kernel(int32_t* counts, long long n) {
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (long long)gridDim.x * 256)
        counts[i] = 0;
}

// alone: this workgroup is the only one and its LDS holds all counters
__global__ __launch_bounds__(256) void balance_count_kernel(BalanceArgs p, int alone) {
    __shared__ int hist[kHist];
    const int lane = threadIdx.x & 63;
    const int t0 = blockIdx.x * kTok, t1 = min(p.T, t0 + kTok);
    int s0 = 0, s1 = p.S - 1;
    if (!alone) {
        s0 = max(sequence_of(p, t0, lane), 0);
        s1 = min(sequence_of(p, t1 - 1, lane), p.S - 1);
    }
    const int per = p.C * p.E;
    const long long need = (long long)max(s1 - s0 + 1, 0) * per;
    const bool lds = need <= kHist;
    if (lds) {
        for (int i = threadIdx.x; i < (int)need; i += 256) hist[i] = 0;
        __syncthreads();
    }
    for (int tb = t0; tb < t1; tb += 256) {
        const int t = tb + threadIdx.x;
        if (t >= t1 || (p.mask && !p.mask[t])) continue;
        int s = 0;
        if (p.offsets) {
            if (t < offset_at(p, 0)) continue;
            // the last of [s0, s1 + 1] whose first token is at or before t
            int lo = s0, hi = s1 + 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (offset_at(p, mid) <= t) lo = mid;
                else hi = mid - 1;
            }
            s = lo;
            if (s > s1 || s >= p.S) continue;
        }
        int e[MOE_MAX_K];
        bool ok = true;
#pragma unroll
        for (int j = 0; j < MOE_MAX_K; ++j)
            if (j < p.k) {
                e[j] = p.ids[(size_t)t * p.k + j];
                ok &= e[j] >= 0 && e[j] < p.E;
            }
        if (!ok) {
            if (p.flags) atomicOr(p.flags, MOE_FLAG_BAD_EXPERT_ID);
            continue;
        }
        const int c = p.C == 2 && p.modality[t] ? p.E : 0;
#pragma unroll
        for (int j = 0; j < MOE_MAX_K; ++j)
            if (j < p.k) {
                if (lds) atomicAdd(&hist[(s - s0) * per + c + e[j]], 1);
                else atomicAdd(p.counts + (size_t)s * per + c + e[j], 1);
            }
    }
    if (!lds) return;
    __syncthreads();
    int32_t* to = p.counts + (size_t)s0 * per;
    for (int i = threadIdx.x; i < (int)need; i += 256) {
        if (alone) to[i] = hist[i];
        else if (hist[i]) atomicAdd(to + i, hist[i]);
    }
}

// What a wave keeps of the group of its tokens: the counts of its lane's
// experts (e = lane + 64 i) for each class, and the groups' tokens.
template <int NPL>
struct Group {
    int s = -2;                            // the sequence (none yet)
    int end = -1;                          // first token behind it
    float c0[NPL], c1[NPL];
    float n0, n1;                          // tokens

    __device__ __forceinline__ void load(const BalanceArgs& p, int seq, int lane) {
        s = seq;
        if (seq < 0 || seq >= p.S) {
            end = seq < 0 ? offset_at(p, 0) : 0x7fffffff;
            return;
        }
        end = offset_at(p, seq + 1);
        const int32_t* c = p.counts + (size_t)seq * p.C * p.E;
        double sum0 = 0.0, sum1 = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 64 * i;
            const int a = e < p.E ? c[e] : 0;
            const int b = e < p.E && p.C == 2 ? c[p.E + e] : 0;
            c0[i] = (float)a;
            c1[i] = (float)b;
            sum0 += a;
            sum1 += b;
        }
        n0 = (float)(wave_sum(sum0) / p.k);
        n1 = (float)(wave_sum(sum1) / p.k);
    }
};

// A token's row: its lane's scores and e (S = 1 / (1 + e)), and the two sums
template <int NPL, bool GRAD>
__global__ __launch_bounds__(256) void balance_rows_kernel(BalanceArgs p, int per_wave) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long first = ((long long)blockIdx.x * 4 + wave) * per_wave;
    if (first >= p.T) return;
    const int t1 = (int)min((long long)p.T, first + per_wave);
    Group<NPL> g;
    for (int t = (int)first; t < t1; ++t) {
        float lv[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            lv[i] = p.logits[(size_t)t * p.E + min(lane + 64 * i, p.E - 1)];
        if (g.s == -2 || t >= g.end) g.load(p, sequence_of(p, t, lane), lane);
        const bool part = g.s >= 0 && g.s < p.S && !(p.mask && !p.mask[t]) && ids_valid(p, t);
        const bool second = p.C == 2 && p.modality[t];
        float s[NPL], e[NPL], sum = 0.0f, cs = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            e[i] = score_exp(lv[i]);
            s[i] = lane + 64 * i < p.E ? 1.0f / (1.0f + e[i]) : 0.0f;
            sum += s[i];
            cs = __builtin_fmaf(second ? g.c1[i] : g.c0[i], s[i], cs);
        }
        sum = wave_sum_f32(sum);
        cs = wave_sum_f32(cs);
        const float q = cs / sum;
        if constexpr (!GRAD) {
            if (lane == 0) p.q[t] = part ? q : -1.0f;
        } else {
            const float n = second ? g.n1 : g.n0;
            const float up = part ? p.d_loss[g.s * p.C + second] / n *
                                        ((float)p.E / ((float)p.k * n)) / sum
                                  : 0.0f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int x = lane + 64 * i;
                if (x >= p.E) continue;
                float d = part ? up * ((second ? g.c1[i] : g.c0[i]) - q) * s[i] * (e[i] * s[i])
                               : 0.0f;
                const size_t at = (size_t)t * p.E + x;
                if (p.add) d += p.add[at];
                p.d_logits[at] = d;
            }
        }
    }
}

// loss of the groups of one sequence: means of q, in 64 bits
__global__ __launch_bounds__(1024) void balance_mean_kernel(BalanceArgs p) {
    __shared__ double sum[16][2];
    __shared__ int num[16][2];
    const int s = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lo = offset_at(p, s), hi = offset_at(p, s + 1);
    double a[2] = {0.0, 0.0};
    int n[2] = {0, 0};
    for (int t = lo + (int)threadIdx.x; t < hi; t += (int)blockDim.x) {
        const float q = p.q[t];
        if (q < 0.0f) continue;
        const int c = p.C == 2 && p.modality[t] ? 1 : 0;
        a[0] += c ? 0.0 : (double)q;
        a[1] += c ? (double)q : 0.0;
        n[0] += !c;
        n[1] += c;
    }
    for (int c = 0; c < 2; ++c) {
        a[c] = wave_sum(a[c]);
        n[c] = wave_scan(n[c], lane);
        if (lane == 63) sum[wave][c] = a[c], num[wave][c] = n[c];
    }
    __syncthreads();
    if ((int)threadIdx.x < p.C) {
        double v = 0.0;
        int m = 0;
        for (int w = 0; w < (int)(blockDim.x >> 6); ++w)
            v += sum[w][threadIdx.x], m += num[w][threadIdx.x];
        p.loss[s * p.C + threadIdx.x] =
            m > 0 ? (float)(v * p.E / ((double)p.k * m) / m) : 0.0f;
    }
}

template <bool GRAD>
hipError_t launch_rows(const BalanceArgs& p, hipStream_t stream) {
    // (consecutive tokens a wave: a group's counts are loaded once for them)
    // (and at most 2^20 workgroups)
    const int per = p.T < 8192 ? 1 : p.T < 16384 ? 2 : p.T <= 1 << 24 ? 4 : 1 + (p.T >> 22);
    const dim3 grid((unsigned)(((long long)p.T + 4 * per - 1) / (4 * per)));
    const int npl = (p.E + 63) / 64;
#define MOE_ROWS(N) \
    hipLaunchKernelGGL((balance_rows_kernel<N, GRAD>), grid, dim3(256), 0, stream, p, per)
    if (npl <= 1) MOE_ROWS(1);
    else if (npl <= 2) MOE_ROWS(2);
    else if (npl <= 4) MOE_ROWS(4);
    else if (npl <= 6) MOE_ROWS(6);
    else if (npl <= 8) MOE_ROWS(8);
    else MOE_ROWS(16);
#undef MOE_ROWS
    return hipGetLastError();
}

}  // namespace

hipError_t launch_balance_loss(const BalanceArgs& p, hipStream_t stream) {
    const long long n = (long long)p.S * p.C * p.E;
    const int alone = p.T <= kTok && n <= kHist;
    if (!alone)
        hipLaunchKernelGGL(balance_zero_kernel, dim3((unsigned)((n + 255) / 256 < 2048 ? (n + 255) / 256 : 2048)),
                           dim3(256), 0, stream, p.counts, n);
    const unsigned groups = (unsigned)(((long long)p.T + kTok - 1) / kTok);
    if (groups || alone)
        hipLaunchKernelGGL(balance_count_kernel, dim3(groups ? groups : 1), dim3(256), 0, stream,
                           p, alone);
    if (p.T > 0) {
        const hipError_t err = launch_rows<false>(p, stream);
        if (err != hipSuccess) return err;
    }
    const int threads = p.T / p.S >= 4096 ? 1024 : 256;
    hipLaunchKernelGGL(balance_mean_kernel, dim3((unsigned)p.S), dim3(threads), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const BalanceArgs& p, hipStream_t stream) {
    if (p.T == 0) return hipSuccess;
    return launch_rows<true>(p, stream);
}

}  // namespace moe
