// C ABI of the operators around the layer in a training step (norm, balance
// loss, gradient norm and clipping) and of the MXFP4 operators: argument
// validation (complete before any launch), workspace sizes, launches.
#include <math.h>

#include <algorithm>
#include <vector>

#include "fp4.h"
#include "step.h"

using namespace moe;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
inline bool is_type(int t) { return t == MOE_IN_BF16 || t == MOE_IN_F32; }

int norm_shape(long long rows, int d, double eps) {
    if (rows < 0 || rows > 0x7fffffffll || d < 1) return MOE_ERR_SHAPE;
    if (d % 8 || d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
    if (!(eps >= 0.0) || isinf(eps)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

int balance_shape(int T, int E, int k, int S) {
    if (T < 0 || E < 1 || k < 1 || S < 1) return MOE_ERR_SHAPE;
    if (E > MOE_MAX_E || k > MOE_MAX_K || S > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    if ((long long)T * k >= (1ll << 31)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

bool grad_tensors_ok(const moe_grad_tensor* t, int count) {
    if (count < 0 || (count > 0 && !t)) return false;
    for (int i = 0; i < count; ++i)
        if (t[i].n < 0 || t[i].n >= (1ll << 46) || !is_type(t[i].dtype)) return false;
    return true;
}

long long chunks_of(int64_t n) { return (n + kGradChunk - 1) / kGradChunk; }

int grad_run_checks(const void* plan, size_t plan_bytes, const float* norm, const void* ws,
                    size_t ws_bytes) {
    if (plan_bytes % sizeof(GradChunk)) return MOE_ERR_SHAPE;
    if ((plan_bytes && !plan) || !norm || !ws) return MOE_ERR_NULL;
    if (!aligned(ws, 256) || ws_bytes < MOE_GRAD_WORKSPACE_BYTES) return MOE_ERR_WORKSPACE;
    if (!aligned(plan, 32) || !aligned(norm, 4)) return MOE_ERR_ALIGN;
    return MOE_OK;
}
static_assert(MOE_GRAD_WORKSPACE_BYTES >= kGradParts * sizeof(double), "the partial sums");

}  // namespace

extern "C" {

int moe_add_rms_norm(const void* x, int x_dtype, const void* residual, int res_dtype,
                     const void* w, int w_dtype, long long rows, int d, double eps,
                     void* res_out, uint16_t* y, uint8_t* codes, float* scales, void* stream) {
    const int st = norm_shape(rows, d, eps);
    if (st != MOE_OK) return st;
    if (!is_type(x_dtype) || !is_type(w_dtype) || (residual && !is_type(res_dtype)))
        return MOE_ERR_UNSUPPORTED;
    if (codes && d % 16) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!x || !w || (residual && !res_out) || (!y && !codes) || !codes != !scales)
        return MOE_ERR_NULL;
    const void* al[] = {x, residual, w, residual ? res_out : nullptr, y, codes};
    for (const void* p : al)
        if (!aligned(p, 16)) return MOE_ERR_ALIGN;
    if (!aligned(scales, 4)) return MOE_ERR_ALIGN;
    NormArgs p{};
    p.x = x;
    p.res = residual;
    p.w = w;
    p.res_out = res_out;
    p.y = y;
    p.codes = codes;
    p.scales = scales;
    p.rows = rows;
    p.d = d;
    p.x_f32 = x_dtype == MOE_IN_F32;
    p.res_f32 = res_dtype == MOE_IN_F32;
    p.w_f32 = w_dtype == MOE_IN_F32;
    p.eps = eps;
    return hip_status(launch_add_rms_norm(p, (hipStream_t)stream));
}

size_t moe_rms_norm_backward_workspace_size(long long rows, int d) {
    if (norm_shape(rows, d, 0.0) != MOE_OK) return 0;
    return align256((size_t)std::max(norm_backward_parts(rows, d), 1) * d * sizeof(float));
}

int moe_rms_norm_backward(const void* s, int s_dtype, const void* w, int w_dtype, const void* dy,
                          int dy_dtype, const void* d_res, int res_dtype, long long rows, int d,
                          double eps, void* dx, int dx_dtype, float* dw, void* ws,
                          size_t ws_bytes, void* stream) {
    const int st = norm_shape(rows, d, eps);
    if (st != MOE_OK) return st;
    if (!is_type(s_dtype) || !is_type(w_dtype) || !is_type(dy_dtype) || !is_type(dx_dtype) ||
        (d_res && !is_type(res_dtype)))
        return MOE_ERR_UNSUPPORTED;
    if (!dw || !ws || (rows > 0 && (!s || !w || !dy || !dx))) return MOE_ERR_NULL;
    if (!aligned(ws, 256) || ws_bytes < moe_rms_norm_backward_workspace_size(rows, d))
        return MOE_ERR_WORKSPACE;
    const void* al[] = {s, w, dy, d_res, dx, dw};
    for (const void* p : al)
        if (!aligned(p, 16)) return MOE_ERR_ALIGN;
    NormBwdArgs p{};
    p.s = s;
    p.w = w;
    p.dy = dy;
    p.d_res = d_res;
    p.dx = dx;
    p.dw = dw;
    p.part = (float*)ws;
    p.rows = rows;
    p.d = d;
    p.s_f32 = s_dtype == MOE_IN_F32;
    p.w_f32 = w_dtype == MOE_IN_F32;
    p.dy_f32 = dy_dtype == MOE_IN_F32;
    p.res_f32 = res_dtype == MOE_IN_F32;
    p.dx_f32 = dx_dtype == MOE_IN_F32;
    p.eps = eps;
    return hip_status(launch_rms_norm_backward(p, (hipStream_t)stream));
}

size_t moe_balance_loss_workspace_size(int T, int E, int S, int classes) {
    if (balance_shape(T, E, 1, S) != MOE_OK || classes < 1 || classes > 2) return 0;
    BalanceArgs p{};
    p.T = T;
    p.E = E;
    p.S = S;
    p.C = classes;
    return balance_layout(p, nullptr);
}

int moe_balance_loss(const float* logits, const int32_t* topk_ids, const int32_t* offsets,
                     const uint8_t* modality, const uint8_t* mask, int T, int E, int k, int S,
                     float* loss, int32_t* counts, uint32_t* d_flags, void* ws, size_t ws_bytes,
                     void* stream) {
    const int st = balance_shape(T, E, k, S);
    if (st != MOE_OK) return st;
    if (!offsets && S != 1) return MOE_ERR_NULL;
    if (!loss || !counts || !ws || (T > 0 && (!logits || !topk_ids))) return MOE_ERR_NULL;
    BalanceArgs p{};
    p.logits = logits;
    p.ids = topk_ids;
    p.offsets = offsets;
    p.modality = modality;
    p.mask = mask;
    p.T = T;
    p.E = E;
    p.k = k;
    p.S = S;
    p.C = modality ? 2 : 1;
    p.counts = counts;
    p.loss = loss;
    if (!aligned(ws, 256) || ws_bytes < balance_layout(p, (char*)ws)) return MOE_ERR_WORKSPACE;
    p.flags = d_flags;
    return hip_status(launch_balance_loss(p, (hipStream_t)stream));
}

int moe_balance_loss_backward(const float* logits, const int32_t* topk_ids,
                              const int32_t* offsets, const uint8_t* modality,
                              const uint8_t* mask, const int32_t* counts, const float* d_loss,
                              const float* add, int T, int E, int k, int S, float* d_logits,
                              void* stream) {
    const int st = balance_shape(T, E, k, S);
    if (st != MOE_OK) return st;
    if (!offsets && S != 1) return MOE_ERR_NULL;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_ids || !counts || !d_loss || !d_logits) return MOE_ERR_NULL;
    BalanceArgs p{};
    p.logits = logits;
    p.ids = topk_ids;
    p.offsets = offsets;
    p.modality = modality;
    p.mask = mask;
    p.T = T;
    p.E = E;
    p.k = k;
    p.S = S;
    p.C = modality ? 2 : 1;
    p.counts = const_cast<int32_t*>(counts);   // (read only there)
    p.d_loss = d_loss;
    p.add = add;
    p.d_logits = d_logits;
    return hip_status(launch_balance_loss_backward(p, (hipStream_t)stream));
}

size_t moe_grad_plan_size(const moe_grad_tensor* tensors, int count) {
    if (!grad_tensors_ok(tensors, count)) return 0;
    size_t chunks = 0;
    for (int i = 0; i < count; ++i) chunks += (size_t)chunks_of(tensors[i].n);
    return chunks * sizeof(GradChunk);
}

int moe_grad_plan(const moe_grad_tensor* tensors, int count, void* host_plan, size_t plan_bytes) {
    if (count < 0) return MOE_ERR_SHAPE;
    if (count > 0 && !tensors) return MOE_ERR_NULL;
    for (int i = 0; i < count; ++i) {
        const moe_grad_tensor& t = tensors[i];
        if (t.n < 0 || t.n >= (1ll << 46)) return MOE_ERR_SHAPE;
        if (!is_type(t.dtype)) return MOE_ERR_UNSUPPORTED;
        if (t.n > 0 && (!t.grad || !t.out)) return MOE_ERR_NULL;
        if (!aligned(t.grad, 16) || !aligned(t.out, 16)) return MOE_ERR_ALIGN;
    }
    const size_t need = moe_grad_plan_size(tensors, count);
    if (need && !host_plan) return MOE_ERR_NULL;
    if (plan_bytes != need) return MOE_ERR_SHAPE;
    // outs against each other, and against the grads of other places
    struct Range {
        uintptr_t lo, hi;
        int i;
        bool out;
    };
    try {
        std::vector<Range> r;
        r.reserve(2 * (size_t)count);
        for (int i = 0; i < count; ++i) {
            const moe_grad_tensor& t = tensors[i];
            if (t.n == 0) continue;
            const uintptr_t n = (uintptr_t)t.n * (t.dtype == MOE_IN_F32 ? 4 : 2);
            r.push_back({(uintptr_t)t.out, (uintptr_t)t.out + n, i, true});
            if (t.grad != t.out) r.push_back({(uintptr_t)t.grad, (uintptr_t)t.grad + n, i, false});
        }
        std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
        // the furthest ends so far of outs and of grads
        uintptr_t outs = 0, grads = 0;
        for (const Range& x : r) {
            if (x.lo < outs || (x.out && x.lo < grads)) return MOE_ERR_UNSUPPORTED;
            (x.out ? outs : grads) = std::max(x.out ? outs : grads, x.hi);
        }
    } catch (...) {                        // (no memory for the ranges)
        return MOE_ERR_WORKSPACE;
    }
    GradChunk* c = (GradChunk*)host_plan;
    for (int i = 0; i < count; ++i) {
        const moe_grad_tensor& t = tensors[i];
        const int f32 = t.dtype == MOE_IN_F32;
        for (int64_t at = 0; at < t.n; at += kGradChunk) {
            const size_t byte = (size_t)at * (f32 ? 4 : 2);
            GradChunk v{};
            v.grad = (const char*)t.grad + byte;
            v.out = (char*)t.out + byte;
            v.n = (int)std::min<int64_t>(kGradChunk, t.n - at);
            v.f32 = f32;
            *c++ = v;
        }
    }
    return MOE_OK;
}

int moe_grad_norm(const void* plan, size_t plan_bytes, float* norm, void* ws, size_t ws_bytes,
                  void* stream) {
    const int st = grad_run_checks(plan, plan_bytes, norm, ws, ws_bytes);
    if (st != MOE_OK) return st;
    return hip_status(launch_grad_norm((const GradChunk*)plan,
                                       (long long)(plan_bytes / sizeof(GradChunk)), (double*)ws,
                                       norm, (hipStream_t)stream));
}

int moe_clip_grad_norm(const void* plan, size_t plan_bytes, double max_norm, float* norm, void* ws,
                       size_t ws_bytes, void* stream) {
    if (!(max_norm >= 0.0)) return MOE_ERR_SHAPE;  // also rejects NaN
    const int st = grad_run_checks(plan, plan_bytes, norm, ws, ws_bytes);
    if (st != MOE_OK) return st;
    return hip_status(launch_clip_grad_norm((const GradChunk*)plan,
                                            (long long)(plan_bytes / sizeof(GradChunk)), max_norm,
                                            (double*)ws, norm, (hipStream_t)stream));
}

int moe_quantize_mxfp4(const void* a, int in_dtype, long long rows, int K, uint8_t* codes,
                       uint8_t* scales, void* stream) {
    if (rows < 0 || K < 1 || rows > (1ll << 45) / K) return MOE_ERR_SHAPE;
    if (K % 32 || !is_type(in_dtype)) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!a || !codes || !scales) return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(codes, 16)) return MOE_ERR_ALIGN;
    return hip_status(
        launch_quant_mxfp4(a, in_dtype, rows, K, codes, scales, (hipStream_t)stream));
}

int moe_grouped_gemm_mxfp4(const uint8_t* a4, const uint8_t* a_scale, const int32_t* offsets,
                           int G, int rows, int K, int N, const uint8_t* w4,
                           const uint8_t* w_scale, int out_dtype, void* out, void* stream) {
    constexpr int kMaxSide = 1 << 22;
    if (G < 1 || rows < 0 || K < 32 || N < 16) return MOE_ERR_SHAPE;
    if (G > MOE_MAX_GROUPS || K % 32 || N % 16 || K > kMaxSide || N > kMaxSide)
        return MOE_ERR_UNSUPPORTED;
    if (out_dtype != MOE_OUT_BF16 && out_dtype != MOE_OUT_F32) return MOE_ERR_UNSUPPORTED;
    if ((long long)rows * K >= (1ll << 40) || (long long)rows * N >= (1ll << 40))
        return MOE_ERR_SHAPE;
    // items of the tile loop: 32-bit
    if (((long long)rows / 32 + G) * ((N + 127) / 128) >= (1ll << 31)) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!a4 || !a_scale || !offsets || !w4 || !w_scale || !out) return MOE_ERR_NULL;
    if (!aligned(a4, 16) || !aligned(w4, 16) || !aligned(out, 16)) return MOE_ERR_ALIGN;
    Fp4GemmArgs g{};
    g.a = a4;
    g.as = a_scale;
    g.offsets = offsets;
    g.G = G;
    g.rows = rows;
    g.K = K;
    g.N = N;
    g.w = w4;
    g.ws = w_scale;
    g.out = out;
    return hip_status(
        launch_grouped_gemm_mxfp4(out_dtype == MOE_OUT_F32, g, (hipStream_t)stream));
}

}  // extern "C"
