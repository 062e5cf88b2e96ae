// The whole layer for a few tokens (T <= MOE_FEW_MAX_T): router, routing,
// routed and shared experts, combine, on weights as checkpoints hold them
// ([out, in] row-major, bf16 or 128-block 8-bit codes), activations bf16.
//
// Bound: HBM.  Every weight row that some token uses is read once and takes
// part in a few products; at one token the read of six experts' and the
// shared expert's matrices is tens of microseconds, so launches and
// dependent round trips count as much as the bandwidth.
//
// One kind of work item serves every product of the layer: 16 weight rows
// times the rows' tokens.  The 8 waves of a workgroup split K in pieces of
// 128 bytes (wave w takes pieces w, w + 8, ..., so the workgroup reads 1 KB
// of each row at a time); a wave's load instruction covers 64 bytes of 16
// rows, which is the operand layout of the 16 x 16 x 32 matrix instruction
// (any order of K will do, the same for weights and activations): the
// weights go from memory to the operand registers and are multiplied by up
// to 16 tokens at once.  The waves' 16 x 16 partial sums meet in LDS and are
// added in wave order.
//
// 8-bit weights are decoded to bf16 (exact); a piece is one block of K, its
// sum is multiplied by the block's scale.
#include "fp8_block.h"
#include "few.h"
#include "route_device.h"

namespace moe {
namespace {

constexpr int kThreads = 512;              // 8 waves
constexpr int kTiles = MOE_FEW_MAX_T / 16; // column tiles of 16 tokens
constexpr int kMaxPairs = MOE_FEW_MAX_T * MOE_MAX_K;
static_assert(kMaxPairs <= kThreads, "one thread a (token, slot) pair");

// Values that other workgroups of the same launch read: stored and loaded at
// device scope (past the XCD's own L2, which is not coherent with the other
// seven), a store complete for every XCD once the wave's store counter says
// so.  A device-wide fence instead would write the whole L2 back at every
// item (133 us instead of 12 for the down products of one token).
__device__ __forceinline__ void put_shared(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float get_shared(const float* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// this wave's stores have completed
__device__ __forceinline__ void stores_done() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

struct Lane {
    int tid, lane, wave, r16, grp;         // r16 = lane % 16, grp = lane / 16
};

__device__ __forceinline__ Lane this_lane() {
    Lane l;
    l.tid = threadIdx.x;
    l.lane = l.tid & 63;
    l.wave = __builtin_amdgcn_readfirstlane(l.tid >> 6);
    l.r16 = l.lane & 15;
    l.grp = l.lane >> 4;
    return l;
}

// acc[c] += this wave's share of W[16 rows] x^T for column tile c < ct.
// wrow: this lane's weight row (row r16 of the item); srow: its block scales
// (8-bit weights); x[c]: the activations of column r16 of tile c, NULL where
// the tile has no such column.
template <bool FP8>
__device__ __forceinline__ void strip(const uint8_t* __restrict__ wrow,
                                      const float* __restrict__ srow, int K,
                                      const uint16_t* const (&x)[kTiles], int ct, const Lane& l,
                                      f32x4 (&acc)[kTiles]) {
    constexpr int UK = FP8 ? 128 : 64;     // K a piece (128 bytes of a row)
    constexpr int UB = 4;                  // pieces in flight a wave
    constexpr int XL = FP8 ? 4 : 2;        // 16-byte activation loads a piece
    const int nu = (K + UK - 1) / UK;
    for (int u0 = l.wave; u0 < nu; u0 += 8 * UB) {
        u32x4 w[UB][2];
        float sc[UB];
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const int u = u0 + 8 * i;
            w[i][0] = w[i][1] = u32x4{0u, 0u, 0u, 0u};
            sc[i] = 0.0f;
            if (u < nu) {
                w[i][0] = *(const u32x4*)(wrow + (size_t)u * 128 + 16 * l.grp);
                if (!FP8 || u * UK + 64 < K)   // (K is a multiple of 64)
                    w[i][1] = *(const u32x4*)(wrow + (size_t)u * 128 + 64 + 16 * l.grp);
                if constexpr (FP8) sc[i] = srow[u];
            }
        }
#pragma unroll
        for (int c = 0; c < kTiles; ++c) {
            if (c >= ct) break;
            u32x4 xv[UB][XL];
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                const int u = u0 + 8 * i;
#pragma unroll
                for (int q = 0; q < XL; ++q) xv[i][q] = u32x4{0u, 0u, 0u, 0u};
                if (u < nu && x[c]) {
                    const uint16_t* xp = x[c] + (size_t)u * UK;
                    if constexpr (FP8) {
                        xv[i][0] = *(const u32x4*)(xp + 16 * l.grp);
                        xv[i][1] = *(const u32x4*)(xp + 16 * l.grp + 8);
                        if (u * UK + 64 < K) {
                            xv[i][2] = *(const u32x4*)(xp + 64 + 16 * l.grp);
                            xv[i][3] = *(const u32x4*)(xp + 64 + 16 * l.grp + 8);
                        }
                    } else {
                        xv[i][0] = *(const u32x4*)(xp + 8 * l.grp);
                        xv[i][1] = *(const u32x4*)(xp + 32 + 8 * l.grp);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                if (u0 + 8 * i >= nu) continue;
                if constexpr (FP8) {
                    f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const u32x4 v = w[i][q >> 1];
                        const bf16x8 wv =
                            fp8x8_to_bf16x8(u32x2{v[2 * (q & 1)], v[2 * (q & 1) + 1]}, 1.0f);
                        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            wv, __builtin_bit_cast(bf16x8, xv[i][q]), part, 0, 0, 0);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[c][e] = __builtin_fmaf(part[e], sc[i], acc[c][e]);
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, w[i][q]),
                            __builtin_bit_cast(bf16x8, xv[i][q]), acc[c], 0, 0, 0);
                }
            }
        }
    }
}

// red: [8 waves][ct][16 rows][16 columns].  The row a lane's scale belongs to
// is the row of its weights, but lane l's outputs are rows 4 (l / 16) + e, so
// 8-bit callers pass the scales of the output rows' block (the same for every
// output row of a lane).
__device__ __forceinline__ void put_partials(float* red, const f32x4 (&acc)[kTiles], int ct,
                                             const Lane& l) {
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
        if (c >= ct) break;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            red[((l.wave * ct + c) * 16 + 4 * l.grp + e) * 16 + l.r16] = acc[c][e];
    }
}

__device__ __forceinline__ float sum_partials(const float* red, int ct, int c, int row, int col) {
    float s = red[(c * 16 + row) * 16 + col];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += red[((w * ct + c) * 16 + row) * 16 + col];
    return s;
}

__device__ __forceinline__ void zero_acc(f32x4 (&acc)[kTiles]) {
#pragma unroll
    for (int c = 0; c < kTiles; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

// the 16 rows of a gate/up item: gate rows of features f0 .. f0 + 7, then the
// up rows of the same features
template <bool FP8>
__device__ __forceinline__ void gate_up_strip(const void* gate, const void* up, const float* sg,
                                              const float* su, size_t mat, int f0, int F, int d,
                                              const uint16_t* const (&x)[kTiles], int ct,
                                              const Lane& l, f32x4 (&acc)[kTiles]) {
    constexpr size_t B = FP8 ? 1 : 2;
    const size_t row = (mat * F + f0 + (l.r16 & 7)) * (size_t)d;
    const uint8_t* wrow = (const uint8_t*)(l.r16 < 8 ? gate : up) + row * B;
    const float* srow = nullptr;
    if constexpr (FP8) {
        const int nbf = (F + 127) / 128, nbd = (d + 127) / 128;
        srow = (l.grp < 2 ? sg : su) + (mat * nbf + f0 / 128) * (size_t)nbd;
    }
    strip<FP8>(wrow, srow, d, x, ct, l, acc);
}

// ------------------------------------------------ router and shared expert --
// Items: 16 experts' router rows, then 8 features of the shared expert: none
// depends on the routing.  Workgroup 0 clears the counters of the last kernel.
template <bool FP8>
__global__ __launch_bounds__(kThreads, 2) void few_router_kernel(FewArgs p) {
    extern __shared__ __align__(16) float red[];
    const Lane l = this_lane();
    const int ct = (p.T + 15) / 16;
    const int nr = (p.E + 15) / 16;
    if (blockIdx.x == 0)
        for (int i = l.tid; i < p.d / 16; i += kThreads) p.count[i] = 0u;
    const uint16_t* x[kTiles];
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
        x[c] = 16 * c + l.r16 < p.T ? p.x + (size_t)(16 * c + l.r16) * p.d : nullptr;
    f32x4 acc[kTiles];
    zero_acc(acc);
    const int item = blockIdx.x;
    if (item < nr) {
        const int e = min(16 * item + l.r16, p.E - 1);
        strip<false>((const uint8_t*)(p.w_g + (size_t)e * p.d), nullptr, p.d, x, ct, l, acc);
        put_partials(red, acc, ct, l);
        __syncthreads();
        for (int i = l.tid; i < 256 * ct; i += kThreads) {
            const int row = i & 15, t = i >> 4, en = 16 * item + row;
            if (t < p.T && en < p.E) {
                float v = sum_partials(red, ct, t >> 4, row, t & 15);
                if (p.logit_offset) v += p.logit_offset[en];
                p.logits[(size_t)t * p.E + en] = v;
            }
        }
    } else {
        const int f0 = 8 * (item - nr);
        gate_up_strip<FP8>(p.s_gate, p.s_up, p.s_gate_scale, p.s_up_scale, 0, f0, p.Fs, p.d, x,
                           ct, l, acc);
        put_partials(red, acc, ct, l);
        __syncthreads();
        for (int i = l.tid; i < 128 * ct; i += kThreads) {
            const int f = i & 7, t = i >> 3;
            if (t < p.T) {
                const float g = sum_partials(red, ct, t >> 4, f, t & 15);
                const float u = sum_partials(red, ct, t >> 4, f + 8, t & 15);
                p.hs[(size_t)t * p.Fs + f0 + f] =
                    f32_to_bf16(clamped_swiglu(g, u, p.clamp_limit, p.clamp_mode));
            }
        }
    }
}

// ------------------------------------------------------------------ routing --
// The distinct experts of a batch and their (token, slot) pairs, in LDS.
struct Table {
    int ids[kMaxPairs];
    float w[kMaxPairs];
    int expert[kMaxPairs];       // distinct experts, in order of first use
    int start[kMaxPairs + 1];    // their first entries in pairs
    int pairs[kMaxPairs];        // pair indexes t k + j, grouped by expert
    int first[kMaxPairs];        // (by pair) start of the expert it is the first of
    int scan[8];
    int n;                       // distinct experts
};

template <int NPL>
__device__ __forceinline__ void topk_token(const FewArgs& p, int t, int lane, int& id, float& w) {
    route_topk_wave<NPL>(p.logits + (size_t)t * p.E, p.score_bias,
                         p.modality ? p.modality + t : nullptr, p.E, p.k, p.n_bias, p.scale, lane,
                         id, w);
}

// one wave: the k experts and weights of token t in lanes j < k (the scores,
// ties, sums and refusals of moe_route); returns the flag bits
__device__ __forceinline__ uint32_t route_token(const FewArgs& p, int t, int lane, int& id,
                                                float& w) {
    if (p.mode == MOE_MODE_TOPK) {
        if (p.E <= 64) topk_token<1>(p, t, lane, id, w);
        else if (p.E <= 256) topk_token<4>(p, t, lane, id, w);
        else if (p.E <= 384) topk_token<6>(p, t, lane, id, w);
        else topk_token<MOE_MAX_E / 64>(p, t, lane, id, w);
        return 0u;
    }
    const int tok = p.input_ids[t];
    id = -1;
    w = 0.0f;
    if (tok < 0 || tok >= p.V) return MOE_FLAG_BAD_INPUT_ID;
    if (lane < p.k) id = p.tid2eid[(size_t)tok * p.k + lane];
    if (__builtin_amdgcn_ballot_w64(lane < p.k && (id < 0 || id >= p.E))) {
        id = -1;
        return MOE_FLAG_BAD_EXPERT_ID;
    }
    const float g = lane < p.k ? score_fn(p.logits[(size_t)t * p.E + id]) : 0.0f;
    float sum = lane_read(g, 0);
    for (int j = 1; j < p.k; ++j) sum = sum + lane_read(g, j);
    w = (g / sum) * p.scale;
    return 0u;
}

// every workgroup routes the batch for itself (the logits are in the caches);
// workgroup 0 writes ids and weights out
__device__ __forceinline__ void build_table(const FewArgs& p, const Lane& l, Table& tb) {
    for (int t = l.wave; t < p.T; t += 8) {
        int id;
        float w;
        const uint32_t bad = route_token(p, t, l.lane, id, w);
        if (l.lane < p.k) {
            tb.ids[t * p.k + l.lane] = id;
            tb.w[t * p.k + l.lane] = w;
            if (blockIdx.x == 0) {
                p.ids[t * p.k + l.lane] = id;
                p.w[t * p.k + l.lane] = w;
            }
        }
        if (bad && l.lane == 0 && blockIdx.x == 0 && p.flags) atomicOr(p.flags, bad);
    }
    __syncthreads();
    const int P = p.T * p.k, me = l.tid;
    int id = -1, rank = 0, count = 0, lead = me;
    if (me < P) {
        id = tb.ids[me];
        for (int q = 0; q < P; ++q) {
            const bool same = tb.ids[q] == id;
            count += same;
            if (same && q < me) {
                if (rank == 0) lead = q;
                ++rank;
            }
        }
    }
    const bool lead_here = me < P && id >= 0 && rank == 0;
    // inclusive scan of (1, rows) over the leading pairs
    int x = lead_here ? (1 << 16) | count : 0;
    const int mine = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off, 64);
        if (l.lane >= off) x += y;
    }
    if (l.lane == 63) tb.scan[l.wave] = x;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 8; ++w) {
        if (w < l.wave) before += tb.scan[w];
        total += tb.scan[w];
    }
    const int ex = before + x - mine;
    if (lead_here) {
        tb.expert[ex >> 16] = id;
        tb.start[ex >> 16] = ex & 0xffff;
        tb.first[me] = ex & 0xffff;
    }
    if (me == 0) {
        tb.n = total >> 16;
        tb.start[total >> 16] = total & 0xffff;
    }
    __syncthreads();
    if (me < P && id >= 0) tb.pairs[tb.first[lead] + rank] = me;
    __syncthreads();
}

// ------------------------------------------------------- routed gate and up --
// Items: (expert, 8 features), every token of the expert at once.
template <bool FP8>
__global__ __launch_bounds__(kThreads, 2) void few_gate_up_kernel(FewArgs p) {
    extern __shared__ __align__(16) float red_all[];
    __shared__ Table tb;
    const Lane l = this_lane();
    build_table(p, l, tb);
    const int n = tb.n;
    if (blockIdx.x == 0) {
        // the table, for the last kernel
        for (int i = l.tid; i < kMaxPairs; i += kThreads) {
            if (i < n) p.expert[i] = tb.expert[i];
            if (i <= n) p.start[i] = tb.start[i];
            if (i < tb.start[n]) p.pairs[i] = tb.pairs[i];
        }
        if (l.tid == 0) {
            p.start[n] = tb.start[n];
            *p.n_expert = n;
        }
    }
    const int per = p.F / 8;
    const int buf = 8 * ((p.T * p.k + 15) / 16 < kTiles ? (p.T * p.k + 15) / 16 : kTiles) * 256;
    int parity = 0;
    for (int it = blockIdx.x; it < n * per; it += gridDim.x) {
        const int u = it / per, f0 = (it - u * per) * 8;
        const int e = tb.expert[u], s = tb.start[u], m_all = tb.start[u + 1] - s;
        // (repeated ids of a hash table can give an expert more rows than
        // there are tokens: in runs of MOE_FEW_MAX_T)
        for (int m0 = 0; m0 < m_all; m0 += MOE_FEW_MAX_T) {
            const int m = min(m_all - m0, MOE_FEW_MAX_T), ct = (m + 15) / 16;
            const uint16_t* x[kTiles];
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                x[c] = 16 * c + l.r16 < m
                           ? p.x + (size_t)(tb.pairs[s + m0 + 16 * c + l.r16] / p.k) * p.d
                           : nullptr;
            f32x4 acc[kTiles];
            zero_acc(acc);
            gate_up_strip<FP8>(p.w_gate, p.w_up, p.w_gate_scale, p.w_up_scale, e, f0, p.F, p.d, x,
                               ct, l, acc);
            float* red = red_all + parity * buf;
            parity ^= 1;
            put_partials(red, acc, ct, l);
            __syncthreads();
            for (int i = l.tid; i < 128 * ct; i += kThreads) {
                const int f = i & 7, r = i >> 3;
                if (r < m) {
                    const float g = sum_partials(red, ct, r >> 4, f, r & 15);
                    const float up = sum_partials(red, ct, r >> 4, f + 8, r & 15);
                    p.h[(size_t)tb.pairs[s + m0 + r] * p.F + f0 + f] =
                        f32_to_bf16(clamped_swiglu(g, up, p.clamp_limit, p.clamp_mode));
                }
            }
        }
    }
}

// --------------------------------------------------------- down and combine --
// y[t, o] = shared + sum_j w_j y_j, j in slot order, for 16 outputs o
__device__ __forceinline__ void combine_chunk(const FewArgs& p, int chunk, int tid) {
    const int P = p.T * p.k;
    for (int i = tid; i < p.T * 16; i += kThreads) {
        const int t = i >> 4;
        const size_t o = (size_t)chunk * 16 + (i & 15);
        float e[MOE_MAX_K];
#pragma unroll
        for (int j = 0; j < MOE_MAX_K; ++j)
            e[j] = j < p.k && p.ids[t * p.k + j] >= 0
                       ? get_shared(&p.part[(size_t)(t * p.k + j) * p.d + o]) : 0.0f;
        float v = p.Fs > 0 ? get_shared(&p.part[(size_t)(P + t) * p.d + o]) : 0.0f;
#pragma unroll
        for (int j = 0; j < MOE_MAX_K; ++j)
            if (j < p.k && p.ids[t * p.k + j] >= 0) v = __builtin_fmaf(p.w[t * p.k + j], e[j], v);
        if (p.out_dtype == MOE_OUT_F32)
            ((float*)p.y)[(size_t)t * p.d + o] = v;
        else
            ((uint16_t*)p.y)[(size_t)t * p.d + o] = f32_to_bf16(v);
    }
}

// Items: (expert or the shared one, 16 outputs).  The workgroup that finishes
// an output chunk's last expert adds the experts up: which one that is does
// not change the order of the sum.
template <bool FP8>
__global__ __launch_bounds__(kThreads, 2) void few_down_kernel(FewArgs p) {
    extern __shared__ __align__(16) float red_all[];
    __shared__ int last_sh[2];
    const Lane l = this_lane();
    const int n = *p.n_expert, sh = p.Fs > 0 ? 1 : 0;
    const int per = p.d / 16;
    const int nct = (p.T * p.k + 15) / 16;
    const int buf = 8 * (nct < kTiles ? nct : kTiles) * 256;
    if (n + sh == 0) {                     // nothing adds to y
        for (int c = blockIdx.x; c < per; c += gridDim.x) combine_chunk(p, c, l.tid);
        return;
    }
    int parity = 0;
    for (int it = blockIdx.x; it < (n + sh) * per; it += gridDim.x) {
        const int u = it / per, chunk = it - u * per;
        const bool shared = u == n;
        const int s = shared ? 0 : p.start[u];
        const int m_all = shared ? p.T : p.start[u + 1] - s;
        const int K = shared ? p.Fs : p.F;
        const size_t mat = shared ? 0 : (size_t)p.expert[u];
        const size_t row = (mat * p.d + 16 * chunk + l.r16) * (size_t)K;
        const uint8_t* wrow =
            (const uint8_t*)(shared ? p.s_down : p.w_down) + row * (FP8 ? 1 : 2);
        const float* srow = nullptr;
        if constexpr (FP8) {
            const int nbd = (p.d + 127) / 128, nbk = (K + 127) / 128;
            srow = (shared ? p.s_down_scale : p.w_down_scale) +
                   (mat * nbd + chunk / 8) * (size_t)nbk;
        }
        for (int m0 = 0; m0 < m_all; m0 += MOE_FEW_MAX_T) {
            const int m = min(m_all - m0, MOE_FEW_MAX_T), ct = (m + 15) / 16;
            const uint16_t* x[kTiles];
#pragma unroll
            for (int c = 0; c < kTiles; ++c) {
                const int r = m0 + 16 * c + l.r16;
                x[c] = r - m0 >= m ? nullptr
                       : shared    ? p.hs + (size_t)r * K
                                   : p.h + (size_t)p.pairs[s + r] * K;
            }
            f32x4 acc[kTiles];
            zero_acc(acc);
            strip<FP8>(wrow, srow, K, x, ct, l, acc);
            float* red = red_all + parity * buf;
            parity ^= 1;
            put_partials(red, acc, ct, l);
            __syncthreads();
            for (int i = l.tid; i < 256 * ct; i += kThreads) {
                const int o = i & 15, r = i >> 4;
                if (r < m) {
                    const size_t slot =
                        shared ? (size_t)p.T * p.k + r : (size_t)p.pairs[s + m0 + r];
                    put_shared(&p.part[slot * p.d + 16 * chunk + o],
                               sum_partials(red, ct, r >> 4, o, r & 15));
                }
            }
        }
        stores_done();                     // the partial outputs, before the count
        __syncthreads();
        int* last = &last_sh[parity];
        if (l.tid == 0)
            *last = __hip_atomic_fetch_add(&p.count[chunk], 1u, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(n + sh - 1);
        __syncthreads();
        if (*last) combine_chunk(p, chunk, l.tid);
    }
}

// (up to 64 tokens need more dynamic LDS than the default limit)
template <bool FP8>
hipError_t set_up() {
    static DeviceSetup setup;
    long long a = 0, b = 0;
    return device_setup(setup, a, b, [](int, long long&, long long&) {
        hipError_t e = hipSuccess;
        for (const void* fn : {(const void*)few_gate_up_kernel<FP8>,
                               (const void*)few_down_kernel<FP8>})
            if (e == hipSuccess)
                e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize,
                                        2 * kTiles * 8 * 256 * (int)sizeof(float));
        return e;
    });
}

template <bool FP8>
hipError_t launch(const FewArgs& p, hipStream_t stream) {
    hipError_t e = set_up<FP8>();
    if (e != hipSuccess) return e;
    const int nt_tok = (p.T + 15) / 16;
    const int nt_pair = (p.T * p.k + 15) / 16 < kTiles ? (p.T * p.k + 15) / 16 : kTiles;
    const size_t wave_tile = 8 * 256 * sizeof(float);
    const int grid1 = (p.E + 15) / 16 + (p.Fs > 0 ? p.Fs / 8 : 0);
    hipLaunchKernelGGL(few_router_kernel<FP8>, dim3(grid1), dim3(kThreads), nt_tok * wave_tile,
                       stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int grid = 2 * device_cu_count();
    hipLaunchKernelGGL(few_gate_up_kernel<FP8>, dim3(grid), dim3(kThreads),
                       2 * nt_pair * wave_tile, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(few_down_kernel<FP8>, dim3(grid), dim3(kThreads), 2 * nt_pair * wave_tile,
                       stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few(bool fp8, const FewArgs& p, hipStream_t stream) {
    return fp8 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace moe
