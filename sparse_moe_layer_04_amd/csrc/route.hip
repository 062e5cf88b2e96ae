// Wavefront router: one 64-lane wave per token (top-k), 64/k tokens per wave
// (hash).
//
// MegaGate order ("HyperParallel accelerates DeepSeek-V4.1 ...", section 2.3):
// score -> bias ranking -> Top-K -> score extraction -> normalise -> scale,
// with separate text / vision bias rows; HashRouter variant ("Twinkle x
// Ascend ...", section "FSDP2-4D parallel engine adaptation"): ids from
// tid2eid[input_ids], weights still from the gate logits.
//
// Each lane owns experts e = lane + 64 i.  The ranking key of an expert is
// the order-preserving 32-bit image of its biased score; top-k is k rounds
// of a wave-wide maximum (DPP row operations, then a lane read) over the
// lanes' largest keys, ties between lanes going to the lowest expert index
// (see route_topk_wave).  This translation unit is built with FP
// contraction off: the score function is a fixed sequence of IEEE binary32
// operations.
#include "route_device.h"

namespace moe {
namespace {

constexpr int kMaxPerLane = MOE_MAX_E / 64;

// one wave per token: see route_topk_wave
template <int NPL>
__global__ __launch_bounds__(256) void route_topk_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const uint8_t* __restrict__ modality, int T, int E, int k, int n_bias, float scale,
    int32_t* __restrict__ ids_out, float* __restrict__ w_out) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= T) return;
    int id;
    float w;
    route_topk_wave<NPL>(logits + (size_t)t * E, bias, modality ? modality + t : nullptr, E, k,
                         n_bias, scale, lane, id, w);
    if (lane < k) {
        ids_out[(size_t)t * k + lane] = id;
        w_out[(size_t)t * k + lane] = w;
    }
}

// Hash routing packs P = 64 / k tokens into a wave: lane l < P k holds slot
// j = l % k of token t = P w + l / k, so the three dependent loads (input
// id, table entry, logit) of every slot are in flight at once.  A token
// whose input id is outside [0, V), or any of whose k table entries is
// outside [0, E), gets ids -1 and weights 0 (ballots over the token's lanes).
__global__ __launch_bounds__(256) void route_hash_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ input_ids,
    const int32_t* __restrict__ tid2eid, int T, int E, int k, int V, float scale,
    int32_t* __restrict__ ids_out, float* __restrict__ w_out, uint32_t* __restrict__ flags) {
    const int lane = threadIdx.x & 63;
    const int P = 64 / k;
    const int q = lane / k, j = lane - q * k;
    const int t = (blockIdx.x * 4 + (threadIdx.x >> 6)) * P + q;
    const bool live = q < P && t < T;
    int tok = -1, id = -1;
    if (live) tok = input_ids[t];
    const bool tok_ok = live && tok >= 0 && tok < V;
    if (tok_ok) id = tid2eid[(size_t)tok * k + j];
    const uint64_t seg = ((1ull << k) - 1) << (q * k);  // this token's lanes
    const uint64_t bad_id = __builtin_amdgcn_ballot_w64(tok_ok && (id < 0 || id >= E));
    const bool ok = tok_ok && (bad_id & seg) == 0;
    float g = 0.0f;
    if (ok) g = score_fn(logits[(size_t)t * E + id]);
    // left-to-right fp32 sum of the token's k scores
    const int base = q * k;
    float sum = __shfl(g, base, 64);
    for (int jj = 1; jj < k; ++jj) sum = sum + __shfl(g, base + jj, 64);
    if (live) {
        ids_out[(size_t)t * k + j] = ok ? id : -1;
        w_out[(size_t)t * k + j] = ok ? (g / sum) * scale : 0.0f;
    }
    const bool bad_tok = __builtin_amdgcn_ballot_w64(live && !tok_ok) != 0;
    if (lane == 0 && flags && (bad_tok || bad_id))
        atomicOr(flags, (bad_tok ? MOE_FLAG_BAD_INPUT_ID : 0u) |
                            (bad_id ? MOE_FLAG_BAD_EXPERT_ID : 0u));
}

// Routing backward ("HyperParallel accelerates DeepSeek-V4.1 ...", section
// 2.3, MegaGate: the gradient chain of the gate's normalisation and scaling):
// given dw[t, j] = dLoss/dw_j for the routing weights
//   w_j = scale * g_j / G,  g_j = S(l[t, ids_j]),  G = sum_j g_j,
// the logits' gradient is
//   dl[t, ids_i] = (scale / G) * (dw_i - sum_j dw_j g_j / G) * g_i (1 - g_i)
// and 0 for the E - k experts the token did not select (the choice is
// piecewise constant in the logits; the ranking bias takes no part in w).
// The bracket is evaluated as sum_j g_j (dw_i - dw_j) / G (equal, since
// sum_j g_j = G): no cancellation between dw_i and the weighted mean, and
// exactly 0 when k = 1 or all dw are equal, as the weights are then
// constant.  One wave per token: lane j < k holds slot j; G and the bracket
// are summed in slot order in fp32; then every lane writes its entries
// e = lane + 64 i of the row (each entry written once; an expert listed in
// two slots gets the sum).  A token with an id outside [0, E) gets a zero
// row and sets MOE_FLAG_BAD_EXPERT_ID.
__global__ __launch_bounds__(256) void route_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, int T, int E, int k, float scale, float* __restrict__ dl,
    uint32_t* __restrict__ flags) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;                          // (wave-uniform)
    int id = -1;
    float dwj = 0.0f;
    if (lane < k) {
        id = ids[(size_t)t * k + lane];
        dwj = dw[(size_t)t * k + lane];
    }
    const bool bad = __builtin_amdgcn_ballot_w64(lane < k && (id < 0 || id >= E)) != 0;
    float* out = dl + (size_t)t * E;
    if (bad) {
        for (int e = lane; e < E; e += 64) out[e] = 0.0f;
        if (lane == 0 && flags) atomicOr(flags, MOE_FLAG_BAD_EXPERT_ID);
        return;
    }
    const float g = lane < k ? score_fn(logits[(size_t)t * E + id]) : 0.0f;
    float G = lane_read(g, 0);
    float br = lane_read(g, 0) * (dwj - lane_read(dwj, 0));
    for (int j = 1; j < k; ++j) {
        G = G + lane_read(g, j);
        br = br + lane_read(g, j) * (dwj - lane_read(dwj, j));
    }
    float dlj = 0.0f;
    if (lane < k) {
        const float dg = scale / G * (br / G);
        dlj = dg * (g * (1.0f - g));
    }
    // the k (id, gradient) pairs, wave-uniform, read once for the whole row
    int sid[MOE_MAX_K];
    float sdl[MOE_MAX_K];
#pragma unroll
    for (int j = 0; j < MOE_MAX_K; ++j) {
        sid[j] = j < k ? __builtin_amdgcn_readlane(id, j) : -1;
        sdl[j] = j < k ? lane_read(dlj, j) : 0.0f;
    }
    for (int e = lane; e < E; e += 64) {
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < MOE_MAX_K; ++j)
            if (sid[j] == e) v = v + sdl[j];
        out[e] = v;
    }
}

template <int NPL>
void launch_topk(dim3 grid, const float* logits, const float* bias, const uint8_t* modality,
                 int T, int E, int k, int n_bias, float scale, int32_t* ids, float* w,
                 hipStream_t stream) {
    hipLaunchKernelGGL(route_topk_kernel<NPL>, grid, dim3(256), 0, stream, logits, bias,
                       modality, T, E, k, n_bias, scale, ids, w);
}

}  // namespace

hipError_t launch_route(const float* logits, const float* bias, const uint8_t* modality,
                        const int32_t* input_ids, const int32_t* tid2eid, int T, int E, int k,
                        int n_bias, int V, int mode, float scale, int32_t* ids, float* w,
                        uint32_t* flags, hipStream_t stream) {
    if (T <= 0) return hipSuccess;
    dim3 grid((T + 3) / 4);
    if (mode == MOE_MODE_HASH) {
        const int per_wave = 64 / k;
        const int waves = (T + per_wave - 1) / per_wave;
        hipLaunchKernelGGL(route_hash_kernel, dim3((waves + 3) / 4), dim3(256), 0, stream, logits,
                           input_ids, tid2eid, T, E, k, V, scale, ids, w, flags);
        return hipGetLastError();
    }
    int npl = (E + 63) / 64;
    if (npl <= 1)
        launch_topk<1>(grid, logits, bias, modality, T, E, k, n_bias, scale, ids, w, stream);
    else if (npl <= 2)
        launch_topk<2>(grid, logits, bias, modality, T, E, k, n_bias, scale, ids, w, stream);
    else if (npl <= 4)
        launch_topk<4>(grid, logits, bias, modality, T, E, k, n_bias, scale, ids, w, stream);
    else if (npl <= 6)
        launch_topk<6>(grid, logits, bias, modality, T, E, k, n_bias, scale, ids, w, stream);
    else if (npl <= 8)
        launch_topk<8>(grid, logits, bias, modality, T, E, k, n_bias, scale, ids, w, stream);
    else
        launch_topk<kMaxPerLane>(grid, logits, bias, modality, T, E, k, n_bias, scale, ids, w,
                                 stream);
    return hipGetLastError();
}

hipError_t launch_route_backward(const float* logits, const int32_t* ids, const float* dw,
                                 int T, int E, int k, float scale, float* dl, uint32_t* flags,
                                 hipStream_t stream) {
    if (T <= 0) return hipSuccess;
    hipLaunchKernelGGL(route_backward_kernel, dim3((T + 3) / 4), dim3(256), 0, stream, logits,
                       ids, dw, T, E, k, scale, dl, flags);
    return hipGetLastError();
}

}  // namespace moe
