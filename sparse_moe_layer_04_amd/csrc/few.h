// Arguments of the few-token layer's kernels.
#pragma once

#include "moe_internal.h"

namespace moe {

// workgroups of the experts' kernel, at most; its counters (two kinds, 8 of
// each, a line apart) and flags (a word a workgroup's share)
constexpr int MOE_FEW_MAX_SHARES = 1024;
constexpr int MOE_FEW_SYNC_BYTES = 2 * 8 * 128 + 4 * MOE_FEW_MAX_SHARES;

struct FewArgs {
    int T, d, E, k, F, Fs, mode, n_bias, V;
    float scale, clamp_limit;
    int clamp_mode, out_dtype;
    const uint16_t* x;             // [T, d] bf16
    const int32_t* input_ids;
    const uint8_t* modality;
    const uint16_t* w_g;           // [E, d] bf16
    const float* logit_offset;
    const float* score_bias;
    const int32_t* tid2eid;
    // bf16, or E4M3 codes with fp32 block scales
    const void *w_gate, *w_up, *w_down, *s_gate, *s_up, *s_down;
    const float *w_gate_scale, *w_up_scale, *w_down_scale;
    const float *s_gate_scale, *s_up_scale, *s_down_scale;
    void* y;
    uint32_t* flags;
    // outputs or workspace
    float* logits;                 // [T, E]
    int32_t* ids;                  // [T, k]
    float* w;                      // [T, k]
    uint16_t* hs;                  // [T, Fs] bf16
    uint16_t* h;                   // [T k, F] bf16, by pair
    uint32_t* sync;                // tickets and flags, MOE_FEW_SYNC_BYTES
};

hipError_t launch_few(bool fp8, const FewArgs& p, hipStream_t stream);

}  // namespace moe
