// Balance loss of the router, with per-expert counts, and its gradient.
//
// A group g is the tokens of one sequence and, with a modality, one class.
// With s = S(logits) (the router's scores), p = s / sum_e s, c[g, e] the pairs
// of the group's tokens at expert e, T_g its tokens and f = E c / (k T_g),
//   loss[g] = 1 / T_g sum_e f_e M_e,  M[g, e] = sum over the group's t of p_te,
// so that one pass over the logits makes the column sums M and the counts side
// by side, neither waiting for the other.  The counts are constants, so with
// q_t = sum_e f_e p_te and u = d_loss[g] / T_g
//   d logits[t, j] = u (f_j - q_t) p_j (1 - s_j):
// a second pass over the logits, in which a row's two sums are made from the
// registers that hold it.
//
// Deterministic without atomics on floats: the first pass writes partial sums
// and counts of the pieces into which the chunks of tokens cut the sequences;
// piece (chunk i, sequence s) has place i + s, since going through the tokens
// each new pair has a larger i + s.  The second kernel adds a sequence's
// pieces, in order, and the last of its workgroups the losses' parts.
//
// Bound: the loss reads the logits once, the gradient reads and writes them.
// 131072 tokens x 384 experts in 16 sequences: 63 us (HBM, 3.2 TB/s) and 86 (4.7);
// 8192 x 384: 14.8 and 10.4, 256 x 64: 7.2 and 3.4 (graph replays): two launches
// and a launch, in each of which the waits for offsets, counts, rows and sums follow
// one another.  What bounds the large ones beside the bytes are a row's scores and
// its sums over the wave: a second division a token took the gradient from 87 to
// 99; in few long sequences the pieces, which one workgroup adds up for 64 columns
// (131072 x 384 with one set of inputs: 44 us in 16 sequences, 93 in one).
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
    const int first = offset_at(p, 0);     // (looked at last: its load with the others')
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
    const int s = lo + __popcll(__builtin_amdgcn_ballot_w64(before));
    return t < first ? -1 : s;
}

// e = exp(-x) and S(x) = 1 / (1 + e), within 4 steps of the router's scores
// (same clamp, NaN as -80): exp2 of the rounded product x log2 e, corrected by
// what the rounding took, and the hardware's reciprocal.  A third of the
// instructions of the router's fixed sequence, whose bits are not needed here.
__device__ __forceinline__ float score_of(float x, float& e) {
    x = __builtin_fminf(__builtin_fmaxf(x, -80.0f), 80.0f);
    const float log2e = 0x1.715476p+0f, log2e_lo = 0x1.4ae0cp-26f;   // their sum: log2 e
    const float a = x * -log2e;
    const float r = __builtin_fmaf(x, -log2e_lo, __builtin_fmaf(x, -log2e, -a));
    const float p = __builtin_amdgcn_exp2f(a);
    e = __builtin_fmaf(p, r * 0x1.62e430p-1f, p);                    // 2^r - 1 = r ln 2
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// What a token is made of: its logits (lane l: experts l + 64 i), slot l's
// expert in lane l < k, its class and mask
template <int NPL>
struct Token {
    float lv[NPL];
    int id;
    uint8_t mod, mask;

    __device__ __forceinline__ void load(const BalanceArgs& p, int t, int lane) {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            lv[i] = p.logits[(size_t)t * p.E + min(lane + 64 * i, p.E - 1)];
        id = p.ids[(size_t)t * p.k + min(lane, p.k - 1)];
        mod = p.C == 2 ? p.modality[t] : 0;
        mask = p.mask ? p.mask[t] : 1;
    }
    __device__ __forceinline__ bool bad(const BalanceArgs& p) const {
        return __builtin_amdgcn_ballot_w64(id < 0 || id >= p.E) != 0;
    }
};

// ---- first pass: a workgroup of W waves takes a chunk of p.chunk tokens, each
// wave every W'th token of a piece.  Lane l holds experts l + 64 i.
template <int NPL, int W>
__global__ __launch_bounds__(64 * W) void balance_pieces_kernel(BalanceArgs p) {
    __shared__ float sums[W][2][NPL * 64];
    __shared__ int hist[2][NPL * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int E = p.E, k = p.k;
    // (places beyond a wave's last token may pass 2^31: unsigned)
    const unsigned t0 = blockIdx.x * (unsigned)p.chunk;
    const unsigned t1 = min((unsigned)p.T, t0 + (unsigned)p.chunk);
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < p.S; s += 64 * W) p.ticket[s] = 0;
    for (unsigned tb = t0; tb < t1;) {
        const int s = sequence_of(p, (int)tb, lane);
        if (s >= p.S) break;
        const unsigned te = min(t1, (unsigned)offset_at(p, s < 0 ? 0 : s + 1));
        if (s < 0 || te <= tb) {             // (before the first sequence; never te <= tb
            tb = max(te, tb + 1);            // with offsets in order)
            continue;
        }
        for (int i = threadIdx.x; i < 2 * NPL * 64; i += 64 * W) (&hist[0][0])[i] = 0;
        __syncthreads();
        float m0[NPL], m1[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) m0[i] = m1[i] = 0.0f;
        Token<NPL> next;
        next.load(p, (int)min(tb + wave, te - 1), lane);
        for (unsigned t = tb + wave; t < te; t += W) {
            Token<NPL> a = next;
            next.load(p, (int)min(t + W, te - 1), lane);
            const int c = a.mod ? 1 : 0;
            const bool bad = a.bad(p);
            if (!a.mask || bad) {
                if (a.mask && lane == 0 && p.flags) atomicOr(p.flags, MOE_FLAG_BAD_EXPERT_ID);
                continue;
            }
            if (lane < k) atomicAdd(&hist[c][a.id], 1);
            float sum = 0.0f, e;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                a.lv[i] = lane + 64 * i < E ? score_of(a.lv[i], e) : 0.0f;
                sum += a.lv[i];
            }
            const float inv = 1.0f / wave_sum_f32(sum);
            const float f0 = c ? 0.0f : inv, f1 = c ? inv : 0.0f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                m0[i] = __builtin_fmaf(a.lv[i], f0, m0[i]);
                m1[i] = __builtin_fmaf(a.lv[i], f1, m1[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            sums[wave][0][lane + 64 * i] = m0[i];
            if (p.C == 2) sums[wave][1][lane + 64 * i] = m1[i];
        }
        __syncthreads();
        const size_t to = ((size_t)blockIdx.x + s) * p.C * E;
        for (int x = threadIdx.x; x < p.C * E; x += 64 * W) {
            const int c = x >= E ? 1 : 0, e = x - c * E;
            float v = sums[0][c][e];
#pragma unroll
            for (int w = 1; w < W; ++w) v += sums[w][c][e];
            p.piece_sum[to + x] = v;
            p.piece_num[to + x] = hist[c][e];
        }
        __syncthreads();
        tb = te;
    }
}

// ---- a sequence's pieces added up: a workgroup takes 64 columns (class,
// expert), its four waves every fourth piece; the counts, and the columns' part
// of sum_e c_e M_e and of sum_e c_e.  The last workgroup of a sequence to end
// adds the parts up.
__global__ __launch_bounds__(256) void balance_join_kernel(BalanceArgs p) {
    __shared__ double sum[4][64];
    __shared__ int num[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int s = blockIdx.y * gridDim.x + blockIdx.x;
    if (s >= p.S) return;
    const int slices = gridDim.z, CE = p.C * p.E;
    const int x = blockIdx.z * 64 + lane;
    const int lo = offset_at(p, s), hi = offset_at(p, s + 1);
    double m = 0.0;
    int n = 0;
    if (x < CE && hi > lo) {
        const int i1 = (hi - 1) / p.chunk;
        for (int i = lo / p.chunk + wave; i <= i1; i += 16) {
            float v[4];
            int c[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const size_t at = ((size_t)min(i + 4 * u, i1) + s) * CE + x;
                v[u] = p.piece_sum[at];
                c[u] = p.piece_num[at];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                m += i + 4 * u <= i1 ? (double)v[u] : 0.0;
                n += i + 4 * u <= i1 ? c[u] : 0;
            }
        }
    }
    sum[wave][lane] = m;
    num[wave][lane] = n;
    __syncthreads();
    if (wave == 0) {
        m = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
        n = num[0][lane] + num[1][lane] + num[2][lane] + num[3][lane];
        if (x < CE) p.counts[(size_t)s * CE + x] = n;
        // (a slice may hold experts of both classes)
        for (int c = 0; c < p.C; ++c) {
            const bool mine = x >= c * p.E && x < (c + 1) * p.E;
            const double v = wave_sum(mine ? m * n : 0.0);
            const double pairs = wave_sum(mine ? (double)n : 0.0);
            if (lane == 0) {
                double* to = p.part + (((size_t)s * slices + blockIdx.z) * 2 + c) * 2;
                __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                __hip_atomic_store(to + 1, pairs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        // (the parts have arrived before the ticket is taken)
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        int ticket = 0;
        if (lane == 0)
            ticket = __hip_atomic_fetch_add(p.ticket + s, 1, __ATOMIC_RELAXED,
                                            __HIP_MEMORY_SCOPE_AGENT);
        if (__builtin_amdgcn_readfirstlane(ticket) != slices - 1) return;
        // lane 32 c + i: slice i of class c
        const int c = lane >> 5, i = lane & 31;
        double v = 0.0, pairs = 0.0;
        if (c < p.C && i < slices) {
            double* from = p.part + (((size_t)s * slices + i) * 2 + c) * 2;
            v = __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            pairs = __hip_atomic_load(from + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        for (int d = 0; d < p.C; ++d) {
            const double total = wave_sum(c == d ? v : 0.0);
            const double tokens = wave_sum(c == d ? pairs : 0.0) / p.k;
            if (lane == 0)
                p.loss[s * p.C + d] =
                    tokens > 0.0 ? (float)(total * p.E / (p.k * tokens * tokens)) : 0.0f;
        }
    }
}
static_assert(2 * MOE_MAX_E <= 32 * 64, "a lane a slice and class");

// What a wave keeps of the group of its tokens: the counts of its lane's
// experts (e = lane + 64 i) for each class, and the groups' tokens.
template <int NPL>
struct Group {
    int s = -2;                            // the sequence (none yet)
    int end = -1;                          // first token behind it
    float c0[NPL], c1[NPL];
    float a0, a1;                          // d_loss / T_g * E / (k T_g)

    // (0 for a group of no pairs, which no token is in)
    __device__ __forceinline__ static float factor(const BalanceArgs& p, float d_loss,
                                                   double pairs) {
        const double n = pairs / p.k;
        return pairs > 0.0 ? (float)((double)d_loss * p.E / (p.k * n * n)) : 0.0f;
    }
    __device__ __forceinline__ void load(const BalanceArgs& p, int seq, int lane) {
        s = seq;
        if (seq < 0 || seq >= p.S) {
            end = seq < 0 ? offset_at(p, 0) : 0x7fffffff;
            return;
        }
        end = offset_at(p, seq + 1);
        const int32_t* c = p.counts + (size_t)seq * p.C * p.E;
        const float u0 = p.d_loss[seq * p.C], u1 = p.d_loss[seq * p.C + p.C - 1];
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
        a0 = factor(p, u0, wave_sum(sum0));
        a1 = p.C == 2 ? factor(p, u1, wave_sum(sum1)) : 0.0f;
    }
};

// ---- the gradient: a wave takes consecutive tokens
template <int NPL>
__global__ __launch_bounds__(256) void balance_gradient_kernel(BalanceArgs p, int per_wave) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long first = ((long long)blockIdx.x * 4 + wave) * per_wave;
    if (first >= p.T) return;
    const int t1 = (int)min((long long)p.T, first + per_wave);
    Token<NPL> next;
    next.load(p, (int)first, lane);
    Group<NPL> g;
    for (int t = (int)first; t < t1; ++t) {
        const Token<NPL> a = next;
        next.load(p, min(t + 1, t1 - 1), lane);
        if (g.s == -2 || t >= g.end) g.load(p, sequence_of(p, t, lane), lane);
        const bool part = g.s >= 0 && g.s < p.S && a.mask && !a.bad(p);
        const bool second = a.mod;
        float s[NPL], e[NPL], sum = 0.0f, cs = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            s[i] = score_of(a.lv[i], e[i]);
            s[i] = lane + 64 * i < p.E ? s[i] : 0.0f;
            sum += s[i];
            cs = __builtin_fmaf(second ? g.c1[i] : g.c0[i], s[i], cs);
        }
        sum = wave_sum_f32(sum);
        cs = wave_sum_f32(cs);
        // (the scores are divided by their sum before they meet d_loss: 1 / sum is
        // up to 5e34, and their product would pass fp32)
        const float inv = 1.0f / sum, q = cs * inv;
        const float up = second ? g.a1 : g.a0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int x = lane + 64 * i;
            if (x >= p.E) continue;
            const float v = up * ((second ? g.c1[i] : g.c0[i]) - q);
            float d = part ? v * (s[i] * inv) * (e[i] * s[i]) : 0.0f;
            const size_t at = (size_t)t * p.E + x;
            if (p.add) d += p.add[at];
            p.d_logits[at] = d;
        }
    }
}

// Tokens of a chunk: enough chunks for every CU, the pieces a small part of
// what is read, and at most 2^18 chunks.  The loss, 8192 tokens x 384 experts:
// 14.6 us with 32 (four waves a workgroup 16.5), 17.1 with 16, 16.4 with 64;
// 32767 x 330: 24.3 us with 32, 22.6 with 64; 131072 x 384: 73 and 61.
int chunk_of(int T) { return T <= 16384 ? 32 : T <= 1 << 24 ? 64 : 2 * (1 + (T >> 19)); }
int slices_of(const BalanceArgs& p) { return (p.C * p.E + 63) / 64; }

#define MOE_BY_EXPERTS(E, CALL)        \
    {                                  \
        const int npl = (E + 63) / 64; \
        if (npl <= 1) CALL(1);         \
        else if (npl <= 2) CALL(2);    \
        else if (npl <= 4) CALL(4);    \
        else if (npl <= 6) CALL(6);    \
        else if (npl <= 8) CALL(8);    \
        else CALL(16);                 \
    }

}  // namespace

size_t balance_layout(BalanceArgs& p, char* base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* q = base ? base + off : nullptr;
        off += (bytes + 255) & ~size_t(255);
        return (void*)q;
    };
    p.chunk = chunk_of(p.T);
    const size_t places = (size_t)((long long)p.T + p.chunk - 1) / p.chunk + p.S;
    p.piece_sum = (float*)take(places * p.C * p.E * 4);
    p.piece_num = (int*)take(places * p.C * p.E * 4);
    p.part = (double*)take((size_t)p.S * slices_of(p) * 4 * 8);
    p.ticket = (int*)take((size_t)p.S * 4);
    return off;
}

hipError_t launch_balance_loss(const BalanceArgs& p, hipStream_t stream) {
    // (a workgroup with T = 0 too: it clears the tickets)
    const unsigned chunks = (unsigned)(((long long)p.T + p.chunk - 1) / p.chunk);
    const dim3 grid(chunks ? chunks : 1);
    // (eight waves a workgroup; four where their sums pass 64 KB of LDS)
#define MOE_PIECES(N)                                                                       \
    hipLaunchKernelGGL((balance_pieces_kernel<N, N <= 8 ? 8 : 4>), grid,                    \
                       dim3(64 * (N <= 8 ? 8 : 4)), 0, stream, p)
    MOE_BY_EXPERTS(p.E, MOE_PIECES)
#undef MOE_PIECES
    const unsigned x = (unsigned)(p.S < 32768 ? p.S : 32768);
    hipLaunchKernelGGL(balance_join_kernel, dim3(x, (unsigned)((p.S + x - 1) / x), slices_of(p)),
                       dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const BalanceArgs& p, hipStream_t stream) {
    if (p.T == 0) return hipSuccess;
    // consecutive tokens a wave, as a group's counts are loaded once for them,
    // but waves for every SIMD (32767 tokens: 51 us with one, 47 with two to
    // four, 46 with eight; 8192: 27.8 with up to two, 30.6 with eight); at most
    // 2^19 workgroups
    const int per = p.T < 4096 ? 1 : p.T <= 16384 ? 2 : p.T <= 1 << 24 ? 8 : 1 + (p.T >> 21);
    const dim3 grid((unsigned)(((long long)p.T + 4 * per - 1) / (4 * per)));
#define MOE_GRADIENT(N) \
    hipLaunchKernelGGL((balance_gradient_kernel<N>), grid, dim3(256), 0, stream, p, per)
    MOE_BY_EXPERTS(p.E, MOE_GRADIENT)
#undef MOE_GRADIENT
    return hipGetLastError();
}

}  // namespace moe
