// C ABI of the 128-block 8-bit operators and of the few-token layer: argument
// validation (complete before any launch), workspace layout, launches.
#include "few.h"
#include "fp8_block.h"

using namespace moe;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// side of a matrix of the 8-bit products (a 256-row tile of codes stays
// within 32-bit offsets)
constexpr int kMaxSide = 1 << 22;

int quant_checks(const void* src, int in_dtype, const uint8_t* codes, const float* scales) {
    if (in_dtype != MOE_IN_BF16 && in_dtype != MOE_IN_F32) return MOE_ERR_UNSUPPORTED;
    if (!src || !codes || !scales) return MOE_ERR_NULL;
    if (!aligned(src, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

int gemm_shape_checks(int G, int rows, int K, int N) {
    if (G < 1 || rows < 0 || K < 16 || N < 16) return MOE_ERR_SHAPE;
    if (G > MOE_MAX_GROUPS || K % 16 || N % 16 || K > kMaxSide || N > kMaxSide)
        return MOE_ERR_UNSUPPORTED;
    if ((long long)rows * K >= (1ll << 40) || (long long)rows * N >= (1ll << 40))
        return MOE_ERR_SHAPE;
    // items of the tile loop: 32-bit
    if (((long long)rows / 128 + G) * block_count(N) >= (1ll << 31)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_quantize_fp8_block(const void* a, int in_dtype, long long rows, int K, uint8_t* codes,
                           float* scales, void* stream) {
    if (rows < 0 || K < 1 || rows > (1ll << 31) || rows * block_count(K) >= (1ll << 31))
        return MOE_ERR_SHAPE;
    if (K % 16) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    const int st = quant_checks(a, in_dtype, codes, scales);
    if (st != MOE_OK) return st;
    return hip_status(
        launch_quant_rows_fp8_block(a, in_dtype, rows, K, codes, scales, (hipStream_t)stream));
}

int moe_quantize_weights_fp8_block(const void* w, int in_dtype, int G, int N, int K,
                                   uint8_t* codes, float* scales, void* stream) {
    if (G < 1 || N < 1 || K < 1) return MOE_ERR_SHAPE;
    if (block_count(N) * block_count(K) >= (1ll << 31) || G * (block_count(N) * block_count(K)) >= (1ll << 31))
        return MOE_ERR_SHAPE;
    if (K % 16) return MOE_ERR_UNSUPPORTED;
    const int st = quant_checks(w, in_dtype, codes, scales);
    if (st != MOE_OK) return st;
    return hip_status(
        launch_quant_matrix_fp8_block(w, in_dtype, G, N, K, codes, scales, (hipStream_t)stream));
}

int moe_grouped_gemm_fp8_block(const uint8_t* a8, const float* a_scale, const int32_t* offsets,
                               int G, int rows, int K, int N, const uint8_t* w8,
                               const float* w_scale, int out_dtype, void* out, void* stream) {
    const int st = gemm_shape_checks(G, rows, K, N);
    if (st != MOE_OK) return st;
    if (out_dtype != MOE_OUT_BF16 && out_dtype != MOE_OUT_F32) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!a8 || !a_scale || !offsets || !w8 || !w_scale || !out) return MOE_ERR_NULL;
    if (!aligned(a8, 16) || !aligned(w8, 16) || !aligned(out, 16) || !aligned(a_scale, 4) ||
        !aligned(w_scale, 4))
        return MOE_ERR_ALIGN;
    Fp8GemmArgs g{};
    g.a = a8;
    g.as = a_scale;
    g.offsets = offsets;
    g.G = G;
    g.rows = rows;
    g.K = K;
    g.N = N;
    g.w1 = w8;
    g.s1 = w_scale;
    g.out = out;
    const bool f32 = out_dtype == MOE_OUT_F32;
    return hip_status(launch_grouped_gemm_fp8_block(f32 ? FP8_OUT_F32 : FP8_OUT_BF16, g,
                                                    (hipStream_t)stream));
}

int moe_expert_ffn_fp8_block(const uint8_t* a8, const float* a_scale, const int32_t* offsets,
                             int G, int rows, int d, int F, const uint8_t* w_gate,
                             const float* w_gate_scale, const uint8_t* w_up,
                             const float* w_up_scale, const uint8_t* w_down,
                             const float* w_down_scale, float clamp_limit, int clamp_mode,
                             uint8_t* h8, float* h_scale, int out_dtype, void* y, void* stream) {
    const int st = gemm_shape_checks(G, rows, d, F);
    if (st != MOE_OK) return st;
    if (!(clamp_limit > 0.0f)) return MOE_ERR_SHAPE;  // also rejects NaN
    if (clamp_mode != MOE_CLAMP_SYMMETRIC && clamp_mode != MOE_CLAMP_GATE_UPPER)
        return MOE_ERR_UNSUPPORTED;
    if (out_dtype != MOE_OUT_BF16 && out_dtype != MOE_OUT_F32) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!a8 || !a_scale || !offsets || !w_gate || !w_gate_scale || !w_up || !w_up_scale ||
        !w_down || !w_down_scale || !h8 || !h_scale || !y)
        return MOE_ERR_NULL;
    if (!aligned(a8, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) ||
        !aligned(h8, 16) || !aligned(y, 16) || !aligned(a_scale, 4) || !aligned(h_scale, 4) ||
        !aligned(w_gate_scale, 4) || !aligned(w_up_scale, 4) || !aligned(w_down_scale, 4))
        return MOE_ERR_ALIGN;
    const bool f32 = out_dtype == MOE_OUT_F32;
    Fp8GemmArgs g{};
    g.a = a8;
    g.as = a_scale;
    g.offsets = offsets;
    g.G = G;
    g.rows = rows;
    g.K = d;
    g.N = F;
    g.w1 = w_gate;
    g.w2 = w_up;
    g.s1 = w_gate_scale;
    g.s2 = w_up_scale;
    g.clamp_limit = clamp_limit;
    g.clamp_mode = clamp_mode;
    g.out = h8;
    g.out_scale = h_scale;
    const hipError_t e = launch_grouped_gemm_fp8_block(FP8_SWIGLU, g, (hipStream_t)stream);
    if (e != hipSuccess) return MOE_ERR_HIP;
    g.a = h8;
    g.as = h_scale;
    g.K = F;
    g.N = d;
    g.w1 = w_down;
    g.s1 = w_down_scale;
    g.out = y;
    return hip_status(launch_grouped_gemm_fp8_block(f32 ? FP8_OUT_F32 : FP8_OUT_BF16, g,
                                                    (hipStream_t)stream));
}

}  // extern "C"

namespace {

// moe_forward_few workspace layout (logits, ids and weights are used where
// the caller takes no copy)
size_t few_layout(const moe_cfg* c, char* base, FewArgs& p) {
    const size_t T = (size_t)c->T, N = T * c->k;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* q = base ? base + off : nullptr;
        off += align256(bytes);
        return (void*)q;
    };
    p.logits = (float*)take(T * c->E * 4);
    p.ids = (int32_t*)take(N * 4);
    p.w = (float*)take(N * 4);
    p.hs = (uint16_t*)take(T * (size_t)(c->F_shared > 0 ? c->F_shared : 0) * 2);
    p.h = (uint16_t*)take(N * c->F * 2);
    p.sync = (uint32_t*)take(MOE_FEW_SYNC_BYTES);
    return off;
}

int few_checks(const moe_cfg* c) {
    if (c->T < 0 || c->E < 1 || c->k < 1 || c->d < 64 || c->F < 64 || c->F_shared < 0)
        return MOE_ERR_SHAPE;
    if (c->T > MOE_FEW_MAX_T) return MOE_ERR_UNSUPPORTED;
    if (c->E > MOE_MAX_E || c->k > MOE_MAX_K || c->k > c->E) return MOE_ERR_UNSUPPORTED;
    if (c->d % 64 || c->F % 64 || c->F_shared % 64) return MOE_ERR_UNSUPPORTED;
    if (c->d > kMaxSide || c->F > kMaxSide || c->F_shared > kMaxSide) return MOE_ERR_UNSUPPORTED;
    if (c->mode != MOE_MODE_TOPK && c->mode != MOE_MODE_HASH) return MOE_ERR_UNSUPPORTED;
    if (c->out_dtype != MOE_OUT_BF16 && c->out_dtype != MOE_OUT_F32) return MOE_ERR_UNSUPPORTED;
    if (!(c->clamp_limit > 0.0f)) return MOE_ERR_SHAPE;
    if (c->clamp_mode != MOE_CLAMP_SYMMETRIC && c->clamp_mode != MOE_CLAMP_GATE_UPPER)
        return MOE_ERR_UNSUPPORTED;
    if (!(c->scale == c->scale)) return MOE_ERR_SHAPE;
    // items of the expert kernels: 32-bit
    if (((long long)c->T * c->k + 1) * (c->F > c->d ? c->F : c->d) >= (1ll << 31))
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_forward_few_workspace_size(const moe_cfg* cfg) {
    if (!cfg || few_checks(cfg) != MOE_OK) return 0;
    FewArgs p{};
    return few_layout(cfg, nullptr, p);
}

int moe_forward_few(const moe_cfg* c, const moe_weights* w, const uint16_t* x,
                    const int32_t* input_ids, const uint8_t* modality, void* y,
                    float* logits_out, int32_t* ids_out, float* w_out, uint32_t* d_flags,
                    void* ws, size_t ws_bytes, void* stream) {
    if (!c || !w) return MOE_ERR_NULL;
    const int st = few_checks(c);
    if (st != MOE_OK) return st;
    const bool fp8 = w->packed == MOE_WEIGHTS_FP8_BLOCK;
    if (w->packed != 0 && !fp8) return MOE_ERR_UNSUPPORTED;
    if (c->T == 0) return MOE_OK;
    if (!x || !y || !w->w_g || !w->w_gate || !w->w_up || !w->w_down) return MOE_ERR_NULL;
    const bool sh = c->F_shared > 0;
    if (sh && (!w->s_gate || !w->s_up || !w->s_down)) return MOE_ERR_NULL;
    if (fp8 && (!w->w_gate_scale || !w->w_up_scale || !w->w_down_scale)) return MOE_ERR_NULL;
    if (fp8 && sh && (!w->s_gate_scale || !w->s_up_scale || !w->s_down_scale))
        return MOE_ERR_NULL;
    if (c->mode == MOE_MODE_TOPK) {
        if (c->n_bias < 0 || c->n_bias > 2) return MOE_ERR_SHAPE;
        if (c->n_bias > 0 && !w->score_bias) return MOE_ERR_NULL;
    } else {
        if (!input_ids || !w->tid2eid) return MOE_ERR_NULL;
        if (c->V < 1) return MOE_ERR_SHAPE;
    }
    if (!ws) return MOE_ERR_NULL;
    FewArgs p{};
    const size_t need = few_layout(c, (char*)ws, p);
    if (!aligned(ws, 256) || ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w->w_g, 16) || !aligned(w->w_gate, 16) ||
        !aligned(w->w_up, 16) || !aligned(w->w_down, 16))
        return MOE_ERR_ALIGN;
    if (sh && (!aligned(w->s_gate, 16) || !aligned(w->s_up, 16) || !aligned(w->s_down, 16)))
        return MOE_ERR_ALIGN;
    if (fp8 && (!aligned(w->w_gate_scale, 4) || !aligned(w->w_up_scale, 4) ||
                !aligned(w->w_down_scale, 4) ||
                (sh && (!aligned(w->s_gate_scale, 4) || !aligned(w->s_up_scale, 4) ||
                        !aligned(w->s_down_scale, 4)))))
        return MOE_ERR_ALIGN;
    p.T = c->T;
    p.d = c->d;
    p.E = c->E;
    p.k = c->k;
    p.F = c->F;
    p.Fs = c->F_shared;
    p.mode = c->mode;
    p.n_bias = c->n_bias;
    p.V = c->V;
    p.scale = c->scale;
    p.clamp_limit = c->clamp_limit;
    p.clamp_mode = c->clamp_mode;
    p.out_dtype = c->out_dtype;
    p.x = x;
    p.input_ids = input_ids;
    p.modality = modality;
    p.w_g = w->w_g;
    p.logit_offset = w->logit_offset;
    p.score_bias = c->n_bias > 0 ? w->score_bias : nullptr;
    p.tid2eid = w->tid2eid;
    p.w_gate = w->w_gate;
    p.w_up = w->w_up;
    p.w_down = w->w_down;
    p.s_gate = w->s_gate;
    p.s_up = w->s_up;
    p.s_down = w->s_down;
    p.w_gate_scale = (const float*)w->w_gate_scale;
    p.w_up_scale = (const float*)w->w_up_scale;
    p.w_down_scale = (const float*)w->w_down_scale;
    p.s_gate_scale = w->s_gate_scale;
    p.s_up_scale = w->s_up_scale;
    p.s_down_scale = w->s_down_scale;
    p.y = y;
    p.flags = d_flags;
    if (logits_out) p.logits = logits_out;
    if (ids_out) p.ids = ids_out;
    if (w_out) p.w = w_out;
    return hip_status(launch_few(fp8, p, (hipStream_t)stream));
}

}  // extern "C"
