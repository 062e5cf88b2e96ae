// The whole layer for a few tokens (T <= MOE_FEW_MAX_T): router, routing,
// routed and shared experts, combine, on weights as checkpoints hold them
// ([out, in] row-major, bf16 or 128-block 8-bit codes), activations bf16.
//
// Bound: HBM.  Every weight row that some token uses is read once and takes
// part in a few products; at one token the read of six experts' and the
// shared expert's matrices is tens of microseconds, so launches and
// dependent round trips count as much as the bandwidth.
//
// One kind of work serves every product of the layer: a strip of 16 weight
// rows times the rows' tokens.  A wave's load instruction covers 64 bytes of
// 16 rows, which is the operand layout of the 16 x 16 x 32 matrix instruction
// (any order of K will do, the same for weights and activations): the weights
// go from memory to the operand registers, eight pieces of 128 bytes a row
// ahead, and are multiplied by up to 16 tokens at once.
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

// The products of a strip: acc[c] += W[16 rows] x^T for column tiles c < ct,
// over the pieces first, first + step, ... of K.
// wrow: this lane's weight row (row r16 of the strip); srow: its block scales
// (8-bit weights); x[c]: the activations of column r16 of tile c (a tile's
// columns past its last token may be anything: no output of theirs is used).
template <bool FP8>
struct Strip {
    static constexpr int UK = FP8 ? 128 : 64;  // K a piece (128 bytes of a row)
    static constexpr int R = 8;                // weight pieces in flight a wave
    static constexpr int RX = 4;               // activation pieces
    static constexpr int XL = FP8 ? 4 : 2;     // 16-byte activation loads a piece

    const uint8_t* wrow;
    const float* srow;
    int K, grp;
    u32x4 w[R][2];
    float sc[R];
    u32x4 xv[RX][XL];

    // piece u; the second half of the last one may lie past K, a multiple of
    // 64: zeros (8-bit)
    __device__ __forceinline__ void load_w(int u, u32x4 (&v)[2], float& s) const {
        const uint8_t* q = wrow + (size_t)u * 128 + 16 * grp;
        v[0] = *(const u32x4*)q;
        if constexpr (FP8) {
            const bool in = u * UK + 64 < K;
            v[1] = *(const u32x4*)(in ? q + 64 : q);
            s = srow[u];
        } else {
            v[1] = *(const u32x4*)(q + 64);
        }
    }
    __device__ __forceinline__ void load_x(const uint16_t* x, int u, u32x4 (&v)[XL]) const {
        const uint16_t* q = x + (size_t)u * UK;
        if constexpr (FP8) {
            v[0] = *(const u32x4*)(q + 16 * grp);
            v[1] = *(const u32x4*)(q + 16 * grp + 8);
            const uint16_t* h = u * UK + 64 < K ? q + 64 : q;
            v[2] = *(const u32x4*)(h + 16 * grp);
            v[3] = *(const u32x4*)(h + 16 * grp + 8);
        } else {
            v[0] = *(const u32x4*)(q + 8 * grp);
            v[1] = *(const u32x4*)(q + 32 + 8 * grp);
        }
    }
    __device__ __forceinline__ void multiply(int u, const u32x4 (&wv)[2], float s,
                                             const u32x4 (&x)[XL], f32x4& acc) const {
        if constexpr (FP8) {
            f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 2; ++q)
                part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    fp8x8_to_bf16x8(u32x2{wv[0][2 * q], wv[0][2 * q + 1]}, 1.0f),
                    __builtin_bit_cast(bf16x8, x[q]), part, 0, 0, 0);
            if (u * UK + 64 < K) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        fp8x8_to_bf16x8(u32x2{wv[1][2 * q], wv[1][2 * q + 1]}, 1.0f),
                        __builtin_bit_cast(bf16x8, x[2 + q]), part, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(part[e], s, acc[e]);
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, wv[q]), __builtin_bit_cast(bf16x8, x[q]), acc, 0, 0,
                    0);
        }
    }
    // pieces first + step * i of K
    __device__ __forceinline__ void run(const uint16_t* const (&x)[kTiles], int ct, int first,
                                        int step, f32x4 (&acc)[kTiles]) {
        const int nu = (K + UK - 1) / UK;
        const int n = first < nu ? (nu - first + step - 1) / step : 0;
        if (ct == 1)
            run_one(x[0], n, first, step, acc[0]);
        else
            run_tiles(x, ct, n, first, step, acc);
    }
    // one column tile: weights R pieces ahead, activations RX
    __device__ __forceinline__ void run_one(const uint16_t* x, int n, int first, int step,
                                            f32x4& acc) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i < n) load_w(first + step * i, w[i], sc[i]);
#pragma unroll
        for (int i = 0; i < RX; ++i)
            if (i < n) load_x(x, first + step * i, xv[i]);
        int i0 = 0;
        for (; i0 + 2 * R <= n; i0 += R) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                multiply(first + step * (i0 + i), w[i], sc[i], xv[i % RX], acc);
                load_w(first + step * (i0 + i + R), w[i], sc[i]);
                load_x(x, first + step * (i0 + i + RX), xv[i % RX]);
            }
        }
        for (; i0 < n; i0 += R) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int k = i0 + i;
                if (k < n) multiply(first + step * k, w[i], sc[i], xv[i % RX], acc);
                if (k + R < n) load_w(first + step * (k + R), w[i], sc[i]);
                if (k + RX < n) load_x(x, first + step * (k + RX), xv[i % RX]);
            }
        }
    }
    // more tokens: each piece against all tiles, the next piece's weights ahead
    __device__ __forceinline__ void run_tiles(const uint16_t* const (&x)[kTiles], int ct, int n,
                                              int first, int step, f32x4 (&acc)[kTiles]) {
        if (n == 0) return;
        load_w(first, w[0], sc[0]);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int u = first + step * i;
            load_w(first + step * min(i + 1, n - 1), w[1], sc[1]);
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                if (c < ct) load_x(x[c], u, xv[c]);
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                if (c < ct) multiply(u, w[0], sc[0], xv[c], acc[c]);
            w[0][0] = w[1][0];
            w[0][1] = w[1][1];
            sc[0] = sc[1];
        }
    }
};
static_assert(Strip<true>::RX >= kTiles && Strip<false>::RX >= kTiles, "a register set a tile");

// A strip whose K is split over the 8 waves: their partial sums meet in LDS,
// red [8 waves][ct][16 rows][16 columns], and are added in wave order.  Lane l
// holds rows 4 (l / 16) + e of column l % 16.
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

// the 16 rows of a gate/up strip: gate rows of features f0 .. f0 + 7, then the
// up rows of the same features.  (A lane's scales are those of its outputs,
// rows 4 (l / 16) + e, not of the row it loads.)
template <bool FP8>
__device__ __forceinline__ void set_gate_up(Strip<FP8>& s, const void* gate, const void* up,
                                            const float* sg, const float* su, size_t mat, int f0,
                                            int F, int d, const Lane& l) {
    const size_t row = (mat * F + f0 + (l.r16 & 7)) * (size_t)d;
    s.wrow = (const uint8_t*)(l.r16 < 8 ? gate : up) + row * (FP8 ? 1 : 2);
    s.K = d;
    s.grp = l.grp;
    if constexpr (FP8) {
        const int nbf = (F + 127) / 128, nbd = (d + 127) / 128;
        s.srow = (l.grp < 2 ? sg : su) + (mat * nbf + f0 / 128) * (size_t)nbd;
    }
}

// ------------------------------------------------ router and shared expert --
// Items: 16 experts' router rows, then 8 features of the shared expert: none
// depends on the routing.  Few strips: each is split over a workgroup's waves.
template <bool FP8>
__global__ __launch_bounds__(kThreads) void few_router_kernel(FewArgs p) {
    extern __shared__ __align__(16) float red[];
    const Lane l = this_lane();
    const int ct = (p.T + 15) / 16;
    const int nr = (p.E + 15) / 16;
    const uint16_t* x[kTiles];
#pragma unroll
    for (int c = 0; c < kTiles; ++c) x[c] = p.x + (size_t)min(16 * c + l.r16, p.T - 1) * p.d;
    f32x4 acc[kTiles];
    zero_acc(acc);
    const int item = blockIdx.x;
    if (item < nr) {
        Strip<false> st;
        st.wrow = (const uint8_t*)(p.w_g + (size_t)min(16 * item + l.r16, p.E - 1) * p.d);
        st.K = p.d;
        st.grp = l.grp;
        st.run(x, ct, l.wave, 8, acc);
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
        Strip<FP8> st;
        set_gate_up(st, p.s_gate, p.s_up, p.s_gate_scale, p.s_up_scale, 0, f0, p.Fs, p.d, l);
        st.run(x, ct, l.wave, 8, acc);
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
// One wave a strip: (expert, 8 features), every token of the expert at once
// (16 columns; more in further column tiles).
template <bool FP8>
__global__ __launch_bounds__(kThreads) void few_gate_up_kernel(FewArgs p) {
    __shared__ Table tb;
    const Lane l = this_lane();
    build_table(p, l, tb);
    const int n = tb.n, P = p.T * p.k;
    if (blockIdx.x == 0) {
        // the table, for the last kernel
        for (int i = l.tid; i < P; i += kThreads) {
            p.expert[i] = tb.expert[i];
            p.pairs[i] = tb.pairs[i];
        }
        for (int i = l.tid; i <= n; i += kThreads) p.start[i] = tb.start[i];
        if (l.tid == 0) *p.n_expert = n;
    }
    const int per = p.F / 8;
    // strips dealt to the workgroups first, so that few strips use every CU
    for (int it = l.wave * gridDim.x + blockIdx.x; it < n * per; it += 8 * gridDim.x) {
        const int u = it / per, f0 = (it - u * per) * 8;
        const int e = tb.expert[u], s = tb.start[u], m_all = tb.start[u + 1] - s;
        // (repeated ids of a hash table can give an expert more rows than
        // there are tokens: in runs of MOE_FEW_MAX_T)
        for (int m0 = 0; m0 < m_all; m0 += MOE_FEW_MAX_T) {
            const int m = min(m_all - m0, MOE_FEW_MAX_T), ct = (m + 15) / 16;
            const uint16_t* x[kTiles];
            int pair[kTiles];
#pragma unroll
            for (int c = 0; c < kTiles; ++c) {
                pair[c] = tb.pairs[s + m0 + min(16 * c + l.r16, m - 1)];
                x[c] = p.x + (size_t)(pair[c] / p.k) * p.d;
            }
            f32x4 acc[kTiles];
            zero_acc(acc);
            Strip<FP8> st;
            set_gate_up(st, p.w_gate, p.w_up, p.w_gate_scale, p.w_up_scale, e, f0, p.F, p.d, l);
            st.run(x, ct, 0, 1, acc);
            // lanes 0-31 hold the gate sums of features 4 grp + e, lanes 32-63
            // the up sums of the same ones
#pragma unroll
            for (int c = 0; c < kTiles; ++c) {
                if (c >= ct) break;
                uint32_t h[2];
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    float v[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mine = acc[c][2 * e2 + i];
                        v[i] = clamped_swiglu(mine, __shfl_xor(mine, 32, 64), p.clamp_limit,
                                              p.clamp_mode);
                    }
                    h[e2] = bf16_pack2(v[0], v[1]);
                }
                if (l.grp < 2 && 16 * c + l.r16 < m)
                    *(u32x2*)(p.h + (size_t)pair[c] * p.F + f0 + 4 * l.grp) = u32x2{h[0], h[1]};
            }
        }
    }
}

// --------------------------------------------------------- down and combine --
// One workgroup 16 outputs, of every expert in turn: its waves take the
// experts (and the shared one) as strips, whose outputs stay in LDS by (token,
// slot) pair until all are there and are then added in slot order, shared
// expert first.  Nothing crosses workgroups, and a token's sum does not depend
// on the batch it is in.
template <bool FP8>
__global__ __launch_bounds__(kThreads) void few_down_kernel(FewArgs p) {
    extern __shared__ __align__(16) float out[];     // [P + T][16]
    __shared__ int expert[kMaxPairs], start[kMaxPairs + 1], pairs[kMaxPairs];
    __shared__ int ids[kMaxPairs], n_sh;
    __shared__ float wt[kMaxPairs];
    const Lane l = this_lane();
    const int P = p.T * p.k, sh = p.Fs > 0 ? 1 : 0;
    // (one round trip: entries past the number of experts are not used)
    if (l.tid < P) {
        expert[l.tid] = p.expert[l.tid];
        start[l.tid] = p.start[l.tid];
        pairs[l.tid] = p.pairs[l.tid];
        ids[l.tid] = p.ids[l.tid];
        wt[l.tid] = p.w[l.tid];
    }
    if (l.tid == 0) {
        start[P] = p.start[P];
        n_sh = *p.n_expert;
    }
    __syncthreads();
    const int n = n_sh;
    for (int chunk = blockIdx.x; chunk < p.d / 16; chunk += gridDim.x) {
        for (int u = l.wave; u < n + sh; u += 8) {
            const bool shared = u >= n;
            const int s = shared ? 0 : start[u];
            const int m_all = shared ? p.T : start[u + 1] - s;
            const int K = shared ? p.Fs : p.F;
            const size_t mat = shared ? 0 : (size_t)expert[u];
            Strip<FP8> st;
            st.wrow = (const uint8_t*)(shared ? p.s_down : p.w_down) +
                      (mat * p.d + 16 * chunk + l.r16) * (size_t)K * (FP8 ? 1 : 2);
            st.K = K;
            st.grp = l.grp;
            if constexpr (FP8) {
                const int nbd = (p.d + 127) / 128, nbk = (K + 127) / 128;
                st.srow = (shared ? p.s_down_scale : p.w_down_scale) +
                          (mat * nbd + chunk / 8) * (size_t)nbk;
            }
            for (int m0 = 0; m0 < m_all; m0 += MOE_FEW_MAX_T) {
                const int m = min(m_all - m0, MOE_FEW_MAX_T), ct = (m + 15) / 16;
                const uint16_t* x[kTiles];
                int slot[kTiles];
#pragma unroll
                for (int c = 0; c < kTiles; ++c) {
                    const int r = m0 + min(16 * c + l.r16, m - 1);
                    slot[c] = shared ? P + r : pairs[s + r];
                    x[c] = shared ? p.hs + (size_t)r * K : p.h + (size_t)slot[c] * K;
                }
                f32x4 acc[kTiles];
                zero_acc(acc);
                st.run(x, ct, 0, 1, acc);
#pragma unroll
                for (int c = 0; c < kTiles; ++c)
                    if (c < ct && 16 * c + l.r16 < m)
                        *(f32x4*)(out + slot[c] * 16 + 4 * l.grp) = acc[c];
            }
        }
        __syncthreads();
        for (int i = l.tid; i < p.T * 16; i += kThreads) {
            const int t = i >> 4, o = i & 15;
            float v = sh ? out[(P + t) * 16 + o] : 0.0f;
            for (int j = 0; j < p.k; ++j)
                if (ids[t * p.k + j] >= 0)
                    v = __builtin_fmaf(wt[t * p.k + j], out[(t * p.k + j) * 16 + o], v);
            const size_t at = (size_t)t * p.d + 16 * chunk + o;
            if (p.out_dtype == MOE_OUT_F32)
                ((float*)p.y)[at] = v;
            else
                ((uint16_t*)p.y)[at] = f32_to_bf16(v);
        }
        __syncthreads();
    }
}

template <bool FP8>
hipError_t launch(const FewArgs& p, hipStream_t stream) {
    const size_t red = (size_t)((p.T + 15) / 16) * 8 * 256 * sizeof(float);
    const int grid1 = (p.E + 15) / 16 + (p.Fs > 0 ? p.Fs / 8 : 0);
    hipLaunchKernelGGL(few_router_kernel<FP8>, dim3(grid1), dim3(kThreads), red, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int cus = device_cu_count();
    hipLaunchKernelGGL(few_gate_up_kernel<FP8>, dim3(cus), dim3(kThreads), 0, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(few_down_kernel<FP8>, dim3(p.d / 16 < cus ? p.d / 16 : cus),
                       dim3(kThreads), (size_t)(p.T * p.k + p.T) * 16 * sizeof(float), stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few(bool fp8, const FewArgs& p, hipStream_t stream) {
    return fp8 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace moe
