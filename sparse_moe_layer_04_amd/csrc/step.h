// Device helpers and launchers of the operators around the layer in a training
// step: the norm with the residual's addition and its backward, the balance
// loss and its gradient, the gradients' norm and their clipping.
#pragma once

#include "fp8_block.h"

namespace moe {

template <int CTRL, int ROWMASK>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWMASK, 0xf, false);
    const int hi =
        __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWMASK, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)lo | (uint64_t)(uint32_t)hi << 32);
}

// Sum of v over the wave, wave-uniform, in a fixed order: pairs, quads, halves
// and rows of 16 lanes, then the rows' sums carried up to lane 63 (lanes that
// a broadcast does not write add zero).
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp_f64<0xB1, 0xf>(v);    // quad_perm [1,0,3,2]
    v += dpp_f64<0x4E, 0xf>(v);    // quad_perm [2,3,0,1]
    v += dpp_f64<0x141, 0xf>(v);   // row_half_mirror
    v += dpp_f64<0x140, 0xf>(v);   // row_mirror
    v += dpp_f64<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
    v += dpp_f64<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const int hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)lo | (uint64_t)(uint32_t)hi << 32);
}

// Eight values of a row in bf16 (16 bytes) or fp32 (32 bytes) as they are in
// memory: loads of several rows are issued together and converted later.
template <bool F32>
struct Raw8 {
    u32x4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, size_t at) {
        const u32x4* q = (const u32x4*)((const uint8_t*)p + at * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = q[i];
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (F32) return __uint_as_float(v[j >> 2][j & 3]);
        const uint32_t u = v[0][j >> 1];
        return __uint_as_float(j & 1 ? u & 0xffff0000u : u << 16);
    }
};
__device__ __forceinline__ u32x4 bf16_pack8(const float (&v)[8]) {
    return u32x4{bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]), bf16_pack2(v[4], v[5]),
                 bf16_pack2(v[6], v[7])};
}
__device__ __forceinline__ void store8(void* p, size_t at, bool f32, const float (&v)[8]) {
    if (f32) {
        *(f32x4*)((float*)p + at) = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4*)((float*)p + at + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *(u32x4*)((uint16_t*)p + at) = bf16_pack8(v);
    }
}

// ----------------------------------------------------------------- host -----
// largest row of the norm
constexpr int kNormMaxD = 16384;

struct NormArgs {
    const void* x;       // [rows, d]
    const void* res;     // [rows, d] or NULL
    const void* w;       // [d]
    void* res_out;       // [rows, d] of res's type (NULL without res)
    uint16_t* y;         // [rows, d] bf16 or NULL
    uint8_t* codes;      // [rows, d] E4M3 or NULL
    float* scales;       // [rows, ceil(d / 128)]
    long long rows;
    int d;
    int x_f32, res_f32, w_f32;
    double eps;
};
hipError_t launch_add_rms_norm(const NormArgs& p, hipStream_t stream);

struct NormBwdArgs {
    const void* s;       // [rows, d] what was normalised
    const void* w;       // [d]
    const void* dy;      // [rows, d]
    const void* d_res;   // [rows, d] or NULL
    void* dx;            // [rows, d]
    float* dw;           // [d]
    float* part;         // [parts, d]
    long long rows;
    int d;
    int s_f32, w_f32, dy_f32, res_f32, dx_f32;
    double eps;
};
int norm_backward_parts(long long rows, int d);
hipError_t launch_rms_norm_backward(const NormBwdArgs& p, hipStream_t stream);

struct BalanceArgs {
    const float* logits;     // [T, E]
    const int32_t* ids;      // [T, k]
    const int32_t* offsets;  // [S + 1] device, or NULL: one sequence of all tokens
    const uint8_t* modality; // [T] or NULL
    const uint8_t* mask;     // [T] or NULL
    int T, E, k, S, C;       // C: classes of tokens (2 with a modality)
    int32_t* counts;         // [S, C, E]
    float* loss;             // [S, C]
    int chunk;               // tokens of a chunk
    float* piece_sum;        // workspace: [chunks + S, C, E] sums of normalised scores
    int* piece_num;          // and pairs of the pieces
    double* part;            // [S, slices, 2, 2]
    int* ticket;             // [S]
    uint32_t* flags;
    const float* d_loss;     // [S, C] (gradient)
    const float* add;        // [T, E] or NULL
    float* d_logits;         // [T, E]
};
// lays the workspace out (sizes are set; base may be NULL): its bytes
size_t balance_layout(BalanceArgs& p, char* base);
hipError_t launch_balance_loss(const BalanceArgs& p, hipStream_t stream);
hipError_t launch_balance_loss_backward(const BalanceArgs& p, hipStream_t stream);

// values of a chunk of the gradients' plan, and its entry
constexpr int kGradChunk = 8192;
struct GradChunk {
    const void* grad;        // the chunk's first value
    void* out;               // where its scaled values go (may be grad)
    int n;                   // values, at most kGradChunk
    int f32;
    int unused[2];
};
static_assert(sizeof(GradChunk) == 32, "one 32-byte load");
// partial sums of squares, at most
constexpr int kGradParts = 2048;
hipError_t launch_grad_norm(const GradChunk* plan, long long chunks, double* part, float* norm,
                            hipStream_t stream);
hipError_t launch_clip_grad_norm(const GradChunk* plan, long long chunks, double max_norm,
                                 double* part, float* norm, hipStream_t stream);

}  // namespace moe
