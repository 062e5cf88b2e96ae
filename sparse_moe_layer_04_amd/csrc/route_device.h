// Wavefront pieces of the routing, shared by the router kernels and the
// few-token layer: the binary32 score function and the top-k of one token.
// (Built with FP contraction off: the score function is a fixed sequence of
// IEEE binary32 operations.)
#pragma once

#include "moe_internal.h"

namespace moe {
namespace {

// Binary32 sigmoid as a fixed operation sequence (see moe.h): clamp to
// [-80, 80] (NaN -> -80); z = -x; n = rint(z * log2 e); Cody-Waite
// r = (z - n*C1) - n*C2 by two fmas with C1 = 0x1.62e4p-1 (exact n*C1) and
// C2 = fl32(ln2 - C1); exp(r) by the degree-7 Taylor polynomial (Horner, fma)
// with binary32 coefficients 1/j!; e = p * 2^n; S = 1 / (1 + e), correctly
// rounded division.
__device__ __forceinline__ float score_fn(float x) {
    x = __builtin_fminf(__builtin_fmaxf(x, -80.0f), 80.0f);  // maxNum: NaN -> -80
    const float log2e = 0x1.715476p+0f;
    const float c1 = 0x1.62e4p-1f;
    const float c2 = 0x1.7f7d1cp-20f;
    float z = -x;
    float t = z * log2e;
    float n = __builtin_rintf(t);
    float r = __builtin_fmaf(-n, c1, z);
    r = __builtin_fmaf(-n, c2, r);
    float p = 0x1.a01a02p-13f;              // 1/5040
    p = __builtin_fmaf(p, r, 0x1.6c16c2p-10f);  // 1/720
    p = __builtin_fmaf(p, r, 0x1.111112p-7f);   // 1/120
    p = __builtin_fmaf(p, r, 0x1.555556p-5f);   // 1/24
    p = __builtin_fmaf(p, r, 0x1.555556p-3f);   // 1/6
    p = __builtin_fmaf(p, r, 0.5f);
    p = __builtin_fmaf(p, r, 1.0f);
    p = __builtin_fmaf(p, r, 1.0f);
    float e = __builtin_ldexpf(p, (int)n);
    float den = 1.0f + e;
    return 1.0f / den;
}

// Order-preserving unsigned image of a binary32 value (finite, no -0):
// negative values have every bit flipped, the others the sign bit set.
__device__ __forceinline__ uint32_t ordered_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// One DPP move; lanes the pattern leaves unwritten get `fill`.
template <int CTRL, int ROWMASK = 0xf>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t fill, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)fill, (int)v, CTRL, ROWMASK, 0xf, false);
}

// Wave-wide maximum (MIN = false) or minimum of v, wave-uniform.  DPP row
// operations only: quad xor 1 and xor 2, half-row and row mirrors leave every
// lane with its 16-lane row's extreme; row broadcasts of lanes 15 and 31
// carry the row extremes up, so lane 63 ends with the wave's, which a lane
// read makes uniform.  Lanes a broadcast does not write see the identity of
// the operation (0 for the maximum, all ones for the minimum).
template <bool MIN>
__device__ __forceinline__ uint32_t wave_reduce_u32(uint32_t v) {
#define MOE_STEP(CTRL, RM)                                   \
    {                                                        \
        const uint32_t o = dpp_u32<CTRL, RM>(MIN ? ~0u : 0u, v); \
        v = MIN ? (o < v ? o : v) : (o > v ? o : v);         \
    }
    MOE_STEP(0xB1, 0xf)    // quad_perm [1,0,3,2]
    MOE_STEP(0x4E, 0xf)    // quad_perm [2,3,0,1]
    MOE_STEP(0x141, 0xf)   // row_half_mirror
    MOE_STEP(0x140, 0xf)   // row_mirror
    MOE_STEP(0x142, 0xa)   // row_bcast:15 into rows 1 and 3
    MOE_STEP(0x143, 0xc)   // row_bcast:31 into rows 2 and 3
#undef MOE_STEP
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// value of lane `src` (wave-uniform) in every lane
__device__ __forceinline__ float lane_read(float v, int src) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), src));
}

// Top-k by (biased score descending, expert index ascending).  Lane l holds
// experts e = l + 64 i (i < NPL) as 32-bit keys (the order-preserving image
// of r; 0 for e >= E, below every real value) with their unbiased scores.
// Round j: m = the wave's largest key (each lane's largest, then a DPP wave
// maximum).  Usually one lane holds m: its keys and scores are read into
// scalar registers and the first i with key m (the lowest expert of that
// lane among equal keys) is the winner.  When several lanes hold m the
// smallest index e among them wins (a wave minimum over each such lane's
// lowest e with key m).  The winner's key is then cleared in its lane.
// All loads of a token (its logits, then the bias row that its modality
// picks) are issued before any score is computed.
// lt: the token's E logits; mod: its modality byte (NULL: bias row 0).  Lane
// j < k returns slot j's expert in id_mine and its weight in w_mine.
template <int NPL>
__device__ __forceinline__ void route_topk_wave(const float* __restrict__ lt,
                                                const float* __restrict__ bias,
                                                const uint8_t* __restrict__ mod, int E, int k,
                                                int n_bias, float scale, int lane, int& id_mine,
                                                float& w_mine) {
    float lv[NPL], bv[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) lv[i] = lt[min(lane + 64 * i, E - 1)];
    if (bias && n_bias > 1 && mod) {
        // both bias rows are loaded beside the modality byte, so the row
        // choice waits for no second round trip
        float b1[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            bv[i] = bias[min(lane + 64 * i, E - 1)];
            b1[i] = bias[E + min(lane + 64 * i, E - 1)];
        }
        if (*mod) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) bv[i] = b1[i];
        }
    } else if (bias) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) bv[i] = bias[min(lane + 64 * i, E - 1)];
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) bv[i] = 0.0f;
    }
    uint32_t key[NPL];
    float sc[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const float s = score_fn(lv[i]);
        const float r = (s + bv[i]) + 0.0f;  // (s > 0: adding a zero bias is exact; -0 -> +0)
        sc[i] = s;
        key[i] = lane + 64 * i < E ? ordered_bits(r) : 0u;
    }
    float g_mine = 0.0f;  // lane j < k keeps g_j
    id_mine = -1;
    for (int j = 0; j < k; ++j) {
        uint32_t lm = key[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) lm = key[i] > lm ? key[i] : lm;
        const uint32_t m = wave_reduce_u32<false>(lm);
        const uint64_t holders = __builtin_amdgcn_ballot_w64(lm == m);
        int w, wi = 0, sbits = 0;  // winner lane, its slot, its score's bits
        if (__popcll(holders) == 1) {
            w = __builtin_ctzll(holders);
#pragma unroll
            for (int i = NPL - 1; i >= 0; --i) {
                const uint32_t kv = (uint32_t)__builtin_amdgcn_readlane((int)key[i], w);
                const int sv = __builtin_amdgcn_readlane(__float_as_int(sc[i]), w);
                if (kv == m) {
                    wi = i;
                    sbits = sv;
                }
            }
        } else {
            uint32_t fe = 0xffffffffu;
#pragma unroll
            for (int i = NPL - 1; i >= 0; --i)
                if (key[i] == m) fe = (uint32_t)(lane + 64 * i);
            const uint32_t e = wave_reduce_u32<true>(fe);
            w = (int)(e & 63);
            wi = (int)(e >> 6);
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (i == wi) sbits = __builtin_amdgcn_readlane(__float_as_int(sc[i]), w);
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (i == wi) key[i] = lane == w ? 0u : key[i];
        if (lane == j) {
            g_mine = __int_as_float(sbits);
            id_mine = w + 64 * wi;
        }
    }
    // left-to-right fp32 sum of the k gathered (unbiased) scores
    float sum = lane_read(g_mine, 0);
    for (int j = 1; j < k; ++j) sum = sum + lane_read(g_mine, j);
    w_mine = (g_mine / sum) * scale;
}

}  // namespace
}  // namespace moe
