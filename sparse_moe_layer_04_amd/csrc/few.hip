// The whole layer for a few tokens (T <= MOE_FEW_MAX_T): router, routing,
// routed and shared experts, combine, on weights as checkpoints hold them
// ([out, in] row-major, bf16 or 128-block 8-bit codes), activations bf16.
//
// Bound: HBM.  Every weight row that some token uses is read once and takes
// part in a few products; at one token the read of six experts' and the
// shared expert's matrices is tens of microseconds, so launches and
// dependent round trips count as much as the bandwidth.  Measured: one token,
// 64 experts of 2048 x 1024, bf16, six and the shared one used: 34 us (88 MB,
// 2.6 TB/s); 384 experts of 4096 x 2048, 8-bit: 58 us (178 MB, 3.1 TB/s);
// eight tokens of those, bf16: 0.40 ms (2.4 GB, 6 TB/s); 33 tokens of them,
// 8-bit: 0.80 ms (3.9 GB, 4.9 TB/s: of an expert with several tokens the
// weights' columns are multiplied once, but every strip reads its tokens'
// activations again).  Of one token's 34 us the first kernel takes 4, the
// second 27: 3 until its workgroups have the experts' table, 12 for the gate
// and up products, 4 until all know that they are done and 7 for the rest; 2
// lie between the kernels.  (Sixteen pieces of the weights in flight for
// eight, or x and h staged in LDS: no faster.  What is asked for earlier in
// the wait makes the wait longer.)
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
constexpr int kMaxPolls = 1 << 22;
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
// over the pieces first, first + STEP, ... of K.
// wrow: this lane's weight row (row r16 of the strip); srow: its block scales
// (8-bit weights); row(c): the activations of column r16 of tile c (a tile's
// columns past its last token may be anything: no output of theirs is used).
template <bool FP8, int STEP>
struct Strip {
    static constexpr int UK = FP8 ? 128 : 64;  // K a piece (128 bytes of a row)
    static constexpr int R = STEP == 1 ? 8 : 4;  // weight pieces in flight a wave
    static constexpr int RX = 4;               // activation pieces
    static constexpr int XL = FP8 ? 4 : 2;     // 16-byte activation loads a piece

    const uint8_t* wrow;
    const float* srow;
    int K, grp;

    static __device__ __forceinline__ void load_w(const uint8_t* q, u32x4 (&v)[2]) {
        v[0] = *(const u32x4*)q;
        v[1] = *(const u32x4*)(q + 64);
    }
    static __device__ __forceinline__ void load_x(const uint16_t* q, u32x4 (&v)[XL]) {
        v[0] = *(const u32x4*)q;
        if constexpr (FP8) {
            v[1] = *(const u32x4*)(q + 8);
            v[2] = *(const u32x4*)(q + 64);
            v[3] = *(const u32x4*)(q + 72);
        } else {
            v[1] = *(const u32x4*)(q + 32);
        }
    }
    // half h of a piece
    static __device__ __forceinline__ void multiply_half(int h, const u32x4& wv,
                                                         const u32x4 (&x)[XL], f32x4& acc) {
        if constexpr (FP8) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    fp8x8_to_bf16x8(u32x2{wv[2 * q], wv[2 * q + 1]}, 1.0f),
                    __builtin_bit_cast(bf16x8, x[2 * h + q]), acc, 0, 0, 0);
        } else {
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv),
                                                          __builtin_bit_cast(bf16x8, x[h]), acc, 0,
                                                          0, 0);
        }
    }
    static __device__ __forceinline__ void multiply(const u32x4 (&wv)[2], float s,
                                                    const u32x4 (&x)[XL], f32x4& acc) {
        if constexpr (FP8) {
            f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
            multiply_half(0, wv[0], x, part);
            multiply_half(1, wv[1], x, part);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(part[e], s, acc[e]);
        } else {
            multiply_half(0, wv[0], x, acc);
            multiply_half(1, wv[1], x, acc);
        }
    }
    // whole pieces of this wave, and whether it has the half piece that a K of
    // an odd number of 64s ends in (8-bit)
    __device__ __forceinline__ int pieces(int first) const {
        const int nu = K / UK;
        return first < nu ? (nu - first + STEP - 1) / STEP : 0;
    }
    __device__ __forceinline__ bool has_half(int first) const {
        return FP8 && K % UK && K / UK % STEP == first % STEP;
    }
    __device__ __forceinline__ void half_piece(const uint16_t* x, f32x4& acc) const {
        const int u = K / UK;
        const u32x4 wv = *(const u32x4*)(wrow + (size_t)u * 128 + 16 * grp);
        u32x4 v[XL];
        const uint16_t* q = x + (size_t)u * UK + 16 * grp;
        v[0] = *(const u32x4*)q;
        v[1] = *(const u32x4*)(q + 8);
        f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
        multiply_half(0, wv, v, part);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(part[e], srow[u], acc[e]);
    }
    // one column tile: weights R pieces ahead, activations RX; ready() returns
    // when the activations may be read
    template <class Ready>
    __device__ __forceinline__ f32x4 run_one(const uint16_t* x, int first,
                                             const Ready& ready) const {
        constexpr int WB = STEP * 128, XB = STEP * UK;   // weight bytes, activations a piece
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        const int n = pieces(first);
        u32x4 w[R][2], xv[RX][XL];
        float sc[R] = {};
        const uint8_t* wq = wrow + (size_t)first * 128 + 16 * grp;
        const uint16_t* xq = x + (size_t)first * UK + (FP8 ? 16 : 8) * grp;
        const float* sq = FP8 ? srow + first : nullptr;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i < n) {
                load_w(wq + i * WB, w[i]);
                if constexpr (FP8) sc[i] = sq[i * STEP];
            }
        ready();
#pragma unroll
        for (int i = 0; i < RX; ++i)
            if (i < n) load_x(xq + i * XB, xv[i]);
        int left = n;
        for (; left >= 2 * R; left -= R) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                multiply(w[i], sc[i], xv[i % RX], acc);
                load_w(wq + (i + R) * WB, w[i]);
                if constexpr (FP8) sc[i] = sq[(i + R) * STEP];
                load_x(xq + (i + RX) * XB, xv[i % RX]);
            }
            wq += R * WB;
            xq += R * XB;
            if constexpr (FP8) sq += R * STEP;
        }
#pragma unroll 1
        for (; left > 0; left -= R) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (i < left) multiply(w[i], sc[i], xv[i % RX], acc);
                if (i + R < left) {
                    load_w(wq + (i + R) * WB, w[i]);
                    if constexpr (FP8) sc[i] = sq[(i + R) * STEP];
                }
                if (i + RX < left) load_x(xq + (i + RX) * XB, xv[i % RX]);
            }
            wq += R * WB;
            xq += R * XB;
            if constexpr (FP8) sq += R * STEP;
        }
        if (has_half(first)) half_piece(x, acc);
        return acc;
    }
    // more tokens: each piece against all tiles, the next piece's weights ahead
    template <class Row>
    __device__ __forceinline__ void run_tiles(const Row& row, int ct, int first,
                                              f32x4 (&acc)[kTiles]) const {
        const int n = pieces(first);
        const uint16_t* x[kTiles];
#pragma unroll
        for (int c = 0; c < kTiles; ++c) {
            x[c] = row(c < ct ? c : 0);
            acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const uint8_t* wq = wrow + (size_t)first * 128 + 16 * grp;
        int at = first * UK + (FP8 ? 16 : 8) * grp;
        u32x4 w[2];
        if (n > 0) load_w(wq, w);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            u32x4 w2[2], xv[kTiles][XL];
            const float s = FP8 ? srow[first + STEP * i] : 0.0f;
            wq += i + 1 < n ? STEP * 128 : 0;
            load_w(wq, w2);
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                if (c < ct) load_x(x[c] + at, xv[c]);
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                if (c < ct) multiply(w, s, xv[c], acc[c]);
            w[0] = w2[0];
            w[1] = w2[1];
            at += STEP * UK;
        }
        if (has_half(first)) {
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                if (c < ct) half_piece(x[c], acc[c]);
        }
    }
    // done(c, sums): called for every tile c < ct
    template <class Row, class Ready, class Done>
    __device__ __forceinline__ void run(const Row& row, int ct, int first, const Ready& ready,
                                        const Done& done) const {
        if (ct == 1) {
            done(0, run_one(row(0), first, ready));
            return;
        }
        ready();
        f32x4 acc[kTiles];
        run_tiles(row, ct, first, acc);
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
            if (c < ct) done(c, acc[c]);
    }
};

// A strip whose K is split over the 8 waves: their partial sums meet in LDS,
// red [8 waves][ct][16 rows][16 columns], and are added in wave order.  Lane l
// holds rows 4 (l / 16) + e of column l % 16.
__device__ __forceinline__ void put_partials(float* red, const f32x4& acc, int c, int ct,
                                             const Lane& l) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        red[((l.wave * ct + c) * 16 + 4 * l.grp + e) * 16 + l.r16] = acc[e];
}

__device__ __forceinline__ float sum_partials(const float* red, int ct, int c, int row, int col) {
    float s = red[(c * 16 + row) * 16 + col];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += red[((w * ct + c) * 16 + row) * 16 + col];
    return s;
}

// the 16 rows of a gate/up strip: gate rows of features f0 .. f0 + 7, then the
// up rows of the same features.  (A lane's scales are those of its outputs,
// rows 4 (l / 16) + e, not of the row it loads.)
template <bool FP8, int STEP>
__device__ __forceinline__ void set_gate_up(Strip<FP8, STEP>& s, const void* gate, const void* up,
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
// (384 experts, d 4096, Fs 2048, 8-bit weights: 24 + 256 items on 256 CUs take
// 10 us.  The router's rows dealt out to the 256 others, two apiece, take 9,
// and one token of the layer 57.8 us for 58.4; two workgroups a CU, 10.)
template <bool FP8>
__global__ __launch_bounds__(kThreads) void few_router_kernel(FewArgs p) {
    extern __shared__ __align__(16) float red[];
    const Lane l = this_lane();
    const int ct = (p.T + 15) / 16;
    const int nr = (p.E + 15) / 16;
    auto row = [&](int c) { return p.x + (size_t)min(16 * c + l.r16, p.T - 1) * p.d; };
    auto partials = [&](int c, const f32x4& acc) { put_partials(red, acc, c, ct, l); };
    const int item = blockIdx.x;
    // the next kernel's counters and flags
    if (item == 0)
        for (int i = l.tid; i < MOE_FEW_SYNC_BYTES / 4; i += kThreads) p.sync[i] = 0u;
    if (item < nr) {
        Strip<false, 8> st;
        st.wrow = (const uint8_t*)(p.w_g + (size_t)min(16 * item + l.r16, p.E - 1) * p.d);
        st.K = p.d;
        st.grp = l.grp;
        st.run(row, ct, l.wave, [] {}, partials);
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
        Strip<FP8, 8> st;
        set_gate_up(st, p.s_gate, p.s_up, p.s_gate_scale, p.s_up_scale, 0, f0, p.Fs, p.d, l);
        st.run(row, ct, l.wave, [] {}, partials);
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
    int lead[MOE_MAX_E];         // (by expert) its first pair, then its first entry
    int scan[8];
    int n;                       // distinct experts
};

template <int NPL>
__device__ __forceinline__ void topk_token(const FewArgs& p, int t, int lane, int& id, float& w) {
    route_topk_wave<NPL>(p.logits + (size_t)t * p.E, p.score_bias,
                         p.modality ? p.modality + t : nullptr, p.E, p.k, p.n_bias, p.scale, lane,
                         id, w);
}

// one wave: the k experts and weights of token t in lanes j < k (top-k)
__device__ __forceinline__ void route_token(const FewArgs& p, int t, int lane, int& id, float& w) {
    if (p.E <= 64) topk_token<1>(p, t, lane, id, w);
    else if (p.E <= 256) topk_token<4>(p, t, lane, id, w);
    else if (p.E <= 384) topk_token<6>(p, t, lane, id, w);
    else topk_token<MOE_MAX_E / 64>(p, t, lane, id, w);
}

// A token takes a wave 2 (up to 64 experts) to 3 us (384), whatever the other
// waves do.  Up to two a wave each workgroup of the experts' kernel routes the
// batch for itself; more get a wave each in a kernel of their own, which costs
// 5 us with its launch.  (32 tokens, 27 experts: 9 us in each workgroup; 31
// tokens, 330 experts: 12.)
constexpr int kOwnTokens = 16;
__host__ __device__ __forceinline__ bool routed_before(const FewArgs& p) {
    return p.mode == MOE_MODE_TOPK && p.T > kOwnTokens;
}
__global__ __launch_bounds__(64) void few_route_kernel(FewArgs p) {
    const int t = blockIdx.x, lane = threadIdx.x;
    int id;
    float w;
    route_token(p, t, lane, id, w);
    if (lane < p.k) {
        p.ids[t * p.k + lane] = id;
        p.w[t * p.k + lane] = w;
    }
}

// ids and weights of the batch into tb (the scores, ties, sums and refusals of
// moe_route); workgroup 0 writes them out
__device__ __forceinline__ void route_batch(const FewArgs& p, const Lane& l, Table& tb) {
    const int P = p.T * p.k, me = l.tid;
    if (p.mode == MOE_MODE_HASH) {
        // a thread a pair
        int id = -1;
        float g = 0.0f;
        if (me < P) {
            const int t = me / p.k, j = me - t * p.k, tok = p.input_ids[t];
            const bool known = tok >= 0 && tok < p.V;
            if (known) id = p.tid2eid[(size_t)tok * p.k + j];
            if (known && (id < 0 || id >= p.E)) id = -2;
            if (id >= 0) g = score_fn(p.logits[(size_t)t * p.E + id]);
            tb.ids[me] = id;
            tb.w[me] = g;
        }
        __syncthreads();
        float w = 0.0f;
        if (me < P) {
            const int first = me / p.k * p.k;
            float sum = 0.0f;
            int worst = 0;
            for (int j = 0; j < p.k; ++j) {
                sum = j ? sum + tb.w[first + j] : tb.w[first];
                worst = min(worst, tb.ids[first + j]);
            }
            w = worst < 0 ? 0.0f : (g / sum) * p.scale;
            id = worst < 0 ? -1 : id;
            if (blockIdx.x == 0) {
                p.ids[me] = id;
                p.w[me] = w;
                if (worst < 0 && me == first && p.flags)
                    atomicOr(p.flags, worst == -2 ? MOE_FLAG_BAD_EXPERT_ID : MOE_FLAG_BAD_INPUT_ID);
            }
        }
        __syncthreads();
        if (me < P) {
            tb.ids[me] = id;
            tb.w[me] = w;
        }
    } else if (routed_before(p)) {
        if (me < P) {
            tb.ids[me] = p.ids[me];
            tb.w[me] = p.w[me];
        }
    } else {
        for (int t = l.wave; t < p.T; t += 8) {
            int id;
            float w;
            route_token(p, t, l.lane, id, w);
            if (l.lane < p.k) {
                tb.ids[t * p.k + l.lane] = id;
                tb.w[t * p.k + l.lane] = w;
                if (blockIdx.x == 0) {
                    p.ids[t * p.k + l.lane] = id;
                    p.w[t * p.k + l.lane] = w;
                }
            }
        }
    }
}

// The table of up to 64 pairs, by one wave: ballots of the ids' bits give each
// pair the set of its expert's pairs.  (One token of the 64-expert layer takes
// 1 us less than with the masks in LDS and their barriers.)
__device__ __forceinline__ void build_small(int P, int lane, Table& tb) {
    static_assert(MOE_MAX_E <= 1 << 10, "bits of an id");
    const int id = lane < P ? tb.ids[lane] : -1;
    uint64_t same = __builtin_amdgcn_ballot_w64(id >= 0);
#pragma unroll
    for (int bit = 0; bit < 10; ++bit) {
        const uint64_t ones = __builtin_amdgcn_ballot_w64(id >> bit & 1);
        same &= id >> bit & 1 ? ones : ~ones;
    }
    if (id < 0) same = 0u;
    const int rank = __popcll(same & ((1ull << lane) - 1u));
    const bool lead_here = id >= 0 && rank == 0;
    // sum of (1, rows) over the leading pairs
    const int mine = lead_here ? (1 << 16) | __popcll(same) : 0, x = wave_scan(mine, lane);
    const int ex = x - mine;
    if (lead_here) {
        tb.expert[ex >> 16] = id;
        tb.start[ex >> 16] = ex & 0xffff;
    }
    const int first = __shfl(ex, same ? __builtin_ctzll(same) : 0, 64) & 0xffff;
    if (id >= 0) tb.pairs[first + rank] = lane;
    if (lane == 63) {
        tb.n = x >> 16;
        tb.start[x >> 16] = x & 0xffff;
    }
}

// The table of more.  mask: P rows of ceil(P / 32) words of LDS.  The first
// pair of an expert has a row with a bit for each of the expert's pairs: their
// number and a pair's place among them are counts of bits.
__device__ __forceinline__ void build_table(const FewArgs& p, const Lane& l, Table& tb,
                                            uint32_t* mask) {
    const int P = p.T * p.k, W = (P + 31) / 32, me = l.tid;
    if (P > 64) {
        for (int i = l.tid; i < P * W; i += kThreads) mask[i] = 0u;
        for (int i = l.tid; i < p.E; i += kThreads) tb.lead[i] = kMaxPairs;
    }
    route_batch(p, l, tb);
    __syncthreads();
    if (P <= 64) {
        if (l.wave == 0) build_small(P, l.lane, tb);
        __syncthreads();
        return;
    }
    const int id = me < P ? tb.ids[me] : -1;
    if (id >= 0) atomicMin(&tb.lead[id], me);
    __syncthreads();
    const int lead = id >= 0 ? tb.lead[id] : 0;
    if (id >= 0) atomicOr(&mask[lead * W + me / 32], 1u << (me % 32));
    __syncthreads();
    int rank = 0, count = 0;
    if (id >= 0)
        for (int i = 0; i < W; ++i) {
            const uint32_t bits = mask[lead * W + i];
            count += __popc(bits);
            rank += __popc(i < me / 32 ? bits : i == me / 32 ? bits & ((1u << (me % 32)) - 1u) : 0u);
        }
    const bool lead_here = id >= 0 && rank == 0;
    const int mine = lead_here ? (1 << 16) | count : 0, x = wave_scan(mine, l.lane);
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
        tb.lead[id] = ex & 0xffff;               // (from here on the first entry)
    }
    if (me == 0) {
        tb.n = total >> 16;
        tb.start[total >> 16] = total & 0xffff;
    }
    __syncthreads();
    if (id >= 0) tb.pairs[tb.lead[id] + rank] = me;
    __syncthreads();
}

// ------------------------------------------------------ the routed experts --
// Gate and up, down and combine in one launch.  Workgroups take work by
// tickets: gridDim.x shares of the gate/up strips first, then the chunks of 16
// outputs.  A chunk needs every share, and a workgroup turns to the chunks
// only once all shares have been taken, by workgroups that are running: who
// waits, waits for work that is going on, however many workgroups the device
// holds at once.  Each of 8 slots (blockIdx % 8, an XCD's workgroups) has its
// own share of the tickets, a line apart: on one counter 256 workgroups queue
// for 16 us.
//
// Gate/up: one wave a strip (expert, 8 features), every token of the expert at
// once (16 columns; more in further column tiles).
// Down: the waves of a workgroup take the experts (and the shared one) of its
// 16 outputs; what they find stays in LDS by (token, slot) pair until all are
// there and is then added in slot order, shared expert first, so that a
// token's sum does not depend on the batch it is in.  The first weights of a
// chunk are on their way while its waves wait for the shares.
//
// h crosses the XCDs, whose L2s are not coherent: it is stored at device scope
// (a fence would write a whole L2 back), its share's flag set once the stores
// have completed, and read after an acquire fence behind the flags.
constexpr int kSlots = 8;
__device__ __forceinline__ uint32_t* sync_word(const FewArgs& p, int kind, int slot) {
    return p.sync + (kind * kSlots + slot) * 32;
}
enum SyncKind : int { kShares = 0, kChunks = 1 };
constexpr int kCounterWords = 2 * kSlots * 32;
static_assert((kCounterWords + MOE_FEW_MAX_SHARES) * 4 == MOE_FEW_SYNC_BYTES,
              "workspace of the counters and flags");
// a word a share: 1 when its h is in memory (a flag each, since additions to
// one counter wait for each other, 60 ns apiece)
__device__ __forceinline__ uint32_t* done_flags(const FewArgs& p) { return p.sync + kCounterWords; }
__device__ __forceinline__ unsigned take(uint32_t* counter) {
    return __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned look(const uint32_t* counter) {
    return __hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// one wave: whether all shares (an even number) are done
__device__ __forceinline__ bool all_done(const FewArgs& p, int shares, int lane) {
    const uint64_t* two = (const uint64_t*)done_flags(p);
    bool open = false;
    for (int i = lane; 2 * i < shares; i += 128) {
        const int j = min(i + 64, shares / 2 - 1);
        const uint64_t a = __hip_atomic_load(two + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint64_t b = __hip_atomic_load(two + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        open |= (a & b) != 0x100000001ull;
    }
    return !__builtin_amdgcn_ballot_w64(open);
}

template <bool FP8>
__global__ __launch_bounds__(kThreads) void few_experts_kernel(FewArgs p) {
    // [P + T][16]; the table's masks before (at most kMaxPairs / 8 = 64 bytes a pair)
    extern __shared__ __align__(16) float out[];
    __shared__ Table tb;
    __shared__ int share_sh, chunk_sh;
    __shared__ unsigned open_sh;
    const Lane l = this_lane();
    const int slot_of = blockIdx.x % kSlots;
    const int shares = gridDim.x, per_slot = shares / kSlots;   // (whole)
    // The last wave takes the tickets (its first thread: a share and, ahead, a
    // chunk): the first ones route, and what a wave loads comes back behind
    // the tickets that it has asked for before, 2 us for 32 of one counter.
    const bool clerk = l.wave == kThreads / 64 - 1;
    unsigned share_t = 0, chunk_t = 0, taken = 0u;
    if (clerk && l.lane == 0) {
        share_t = take(sync_word(p, kShares, slot_of));
        chunk_t = take(sync_word(p, kChunks, slot_of));
        open_sh = 0u;
    }
    bool opened = false;                             // the shares are done
    build_table(p, l, tb, (uint32_t*)out);
    const int n = tb.n, P = p.T * p.k, sh = p.Fs > 0 ? 1 : 0;
    const int per = p.F / 8, strips = n * per;
    // Chunks by 16 outputs and, where those are fewer than the workgroups, by
    // parts of the tokens: a part's experts' weights are read again, from the
    // caches.  (31 tokens, 330 experts, d 256, 8-bit weights: 16 workgroups of
    // 111 experts' strips 19 us, 256 of two tokens' 6; 64 tokens, 64 experts,
    // d 2048: the whole layer 256 us with 128 chunks, 218 with 256.)
    const int columns = p.d / 16;
    const int tokens = (p.T + max(shares / columns, 1) - 1) / max(shares / columns, 1);
    const int chunks = columns * ((p.T + tokens - 1) / tokens);
    bool more_shares = true;
    for (;;) {
        if (more_shares && clerk) {
            // the slot's next share, or one that another slot has left (lane l
            // holds how many of slot l's were taken when it last looked)
            int share = (int)share_t < per_slot ? slot_of + kSlots * (int)share_t : -1;
            share = __builtin_amdgcn_readfirstlane(share);
            while (share < 0) {
                const uint64_t left = __builtin_amdgcn_ballot_w64(l.lane < kSlots &&
                                                                  taken < (unsigned)per_slot);
                if (!left) break;
                const int from = __builtin_ctzll(left);
                unsigned got = 0;
                if (l.lane == 0) got = take(sync_word(p, kShares, from));
                got = (unsigned)__builtin_amdgcn_readfirstlane((int)got);
                if ((int)got < per_slot) share = from + kSlots * (int)got;
                else if (l.lane < kSlots) taken = look(sync_word(p, kShares, l.lane));
            }
            if (l.lane == 0) share_sh = share;
        }
        if (clerk && l.lane == 0) chunk_sh = slot_of + kSlots * (int)min(chunk_t, 1u << 24);
        __syncthreads();
        const int share = more_shares ? share_sh : -1, chunk = chunk_sh;
        more_shares = share >= 0;
        if (more_shares) {
            if (clerk) {
                if (l.lane == 0) share_t = take(sync_word(p, kShares, slot_of));
                if (l.lane < kSlots) taken = look(sync_word(p, kShares, l.lane));
            }
            // (strips dealt to the shares first, so that few strips use every
            // CU; finer shares or strips taken one by one balance the CUs
            // better but end no earlier: memory's rate decides)
            for (int it = l.wave * shares + share; it < strips; it += 8 * shares) {
                const int u = it / per, f0 = (it - u * per) * 8;
                const int e = tb.expert[u], s = tb.start[u], m_all = tb.start[u + 1] - s;
                // (repeated ids of a hash table can give an expert more rows
                // than there are tokens: in runs of MOE_FEW_MAX_T)
                for (int m0 = 0; m0 < m_all; m0 += MOE_FEW_MAX_T) {
                    const int m = min(m_all - m0, MOE_FEW_MAX_T), ct = (m + 15) / 16;
                    auto pair = [&](int c) {
                        return tb.pairs[s + m0 + min(16 * c + l.r16, m - 1)];
                    };
                    Strip<FP8, 1> st;
                    set_gate_up(st, p.w_gate, p.w_up, p.w_gate_scale, p.w_up_scale, e, f0, p.F,
                                p.d, l);
                    // lanes 0-31 hold the gate sums of features 4 grp + i,
                    // lanes 32-63 the up sums of the same ones
                    st.run([&](int c) { return p.x + (size_t)(pair(c) / p.k) * p.d; }, ct, 0,
                           [] {}, [&](int c, const f32x4& acc) {
                               float v[4];
#pragma unroll
                               for (int i = 0; i < 4; ++i)
                                   v[i] = clamped_swiglu(acc[i], __shfl_xor(acc[i], 32, 64),
                                                         p.clamp_limit, p.clamp_mode);
                               const uint64_t h = (uint64_t)bf16_pack2(v[0], v[1]) |
                                                  (uint64_t)bf16_pack2(v[2], v[3]) << 32;
                               if (l.grp < 2 && 16 * c + l.r16 < m)
                                   __hip_atomic_store(
                                       (uint64_t*)(p.h + (size_t)pair(c) * p.F + f0 + 4 * l.grp),
                                       h, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                           });
                }
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's stores are there
            __syncthreads();
            if (l.tid == 0)
                __hip_atomic_store(done_flags(p) + share, 1u, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            continue;
        }
        if (chunk >= chunks) return;
        if (clerk && l.lane == 0) chunk_t = take(sync_word(p, kChunks, slot_of));
        // the clerk watches the flags for all (through LDS: a wave's own load
        // would queue behind its weights)
        auto ready = [&] {
            if (opened) return;
            auto is_open = [&] {
                return __hip_atomic_load(&open_sh, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_WORKGROUP) != 0u;
            };
            if (clerk && !is_open()) {
                // (the limit, seconds, ends the wait when another call has
                // cleared the flags of this call's workspace meanwhile)
                int polls = 0;
                while (!all_done(p, shares, l.lane) && ++polls < kMaxPolls)
                    __builtin_amdgcn_s_sleep(1);
                if (polls == kMaxPolls && l.lane == 0 && p.flags)
                    atomicOr(p.flags, MOE_FLAG_OVERLAP);
                // (for the whole workgroup: its waves share the caches that
                // this invalidates)
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                __hip_atomic_store(&open_sh, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            }
            while (!is_open()) __builtin_amdgcn_s_sleep(1);
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
            opened = true;
        };
        if (clerk) ready();
        const int column = chunk % columns, t0 = chunk / columns * tokens;
        const int t1 = min(t0 + tokens, p.T);
        for (int u = l.wave; u < n + sh; u += 8) {
            const bool shared = u >= n;
            // the part's entries of the expert (they are in the tokens' order)
            int s = shared ? t0 : tb.start[u], m_all = shared ? t1 - t0 : tb.start[u + 1] - s;
            if (!shared && tokens < p.T) {
                int below = 0, inside = 0;
                for (int i = 0; i < m_all; i += 64) {
                    const int q = i + l.lane < m_all ? tb.pairs[s + i + l.lane] : kMaxPairs;
                    below += __popcll(__builtin_amdgcn_ballot_w64(q < t0 * p.k));
                    inside += __popcll(__builtin_amdgcn_ballot_w64(q >= t0 * p.k && q < t1 * p.k));
                }
                s += below;
                m_all = inside;
            }
            const int K = shared ? p.Fs : p.F;
            const size_t mat = shared ? 0 : (size_t)tb.expert[u];
            Strip<FP8, 1> st;
            st.wrow = (const uint8_t*)(shared ? p.s_down : p.w_down) +
                      (mat * p.d + 16 * column + l.r16) * (size_t)K * (FP8 ? 1 : 2);
            st.K = K;
            st.grp = l.grp;
            if constexpr (FP8) {
                const int nbd = (p.d + 127) / 128, nbk = (K + 127) / 128;
                st.srow = (shared ? p.s_down_scale : p.w_down_scale) +
                          (mat * nbd + column / 8) * (size_t)nbk;
            }
            for (int m0 = 0; m0 < m_all; m0 += MOE_FEW_MAX_T) {
                const int m = min(m_all - m0, MOE_FEW_MAX_T), ct = (m + 15) / 16;
                auto slot = [&](int c) {
                    const int r = s + m0 + min(16 * c + l.r16, m - 1);
                    return shared ? P + r : tb.pairs[r];
                };
                st.run([&](int c) { return shared ? p.hs + (size_t)(slot(c) - P) * K
                                                  : p.h + (size_t)slot(c) * K; },
                       ct, 0, ready, [&](int c, const f32x4& acc) {
                           if (16 * c + l.r16 < m)
                               *(f32x4*)(out + slot(c) * 16 + 4 * l.grp) = acc;
                       });
            }
        }
        __syncthreads();
        for (int i = l.tid; i < (t1 - t0) * 16; i += kThreads) {
            const int t = t0 + (i >> 4), o = i & 15;
            float v = sh ? out[(P + t) * 16 + o] : 0.0f;
            for (int j = 0; j < p.k; ++j)
                if (tb.ids[t * p.k + j] >= 0)
                    v = __builtin_fmaf(tb.w[t * p.k + j], out[(t * p.k + j) * 16 + o], v);
            const size_t at = (size_t)t * p.d + 16 * column + o;
            if (p.out_dtype == MOE_OUT_F32)
                ((float*)p.y)[at] = v;
            else
                ((uint16_t*)p.y)[at] = f32_to_bf16(v);
        }
    }
}

template <bool FP8>
hipError_t launch(const FewArgs& p, hipStream_t stream) {
    const size_t red = (size_t)((p.T + 15) / 16) * 8 * 256 * sizeof(float);
    const int grid1 = (p.E + 15) / 16 + (p.Fs > 0 ? p.Fs / 8 : 0);
    hipLaunchKernelGGL(few_router_kernel<FP8>, dim3(grid1), dim3(kThreads), red, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (routed_before(p)) {
        hipLaunchKernelGGL(few_route_kernel, dim3(p.T), dim3(64), 0, stream, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int shares = min((device_cu_count() + 7) & ~7, MOE_FEW_MAX_SHARES);
    hipLaunchKernelGGL(few_experts_kernel<FP8>, dim3(shares), dim3(kThreads),
                       (size_t)(p.T * p.k + p.T) * 16 * sizeof(float), stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few(bool fp8, const FewArgs& p, hipStream_t stream) {
    return fp8 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace moe
