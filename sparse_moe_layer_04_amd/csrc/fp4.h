// Device helpers and launchers of the MXFP4 operators on row-major codes.
#pragma once

#include "fp8_block.h"

namespace moe {

hipError_t launch_quant_mxfp4(const void* a, int in_dtype, long long rows, int K, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream);

struct Fp4GemmArgs {
    const uint8_t* a;        // [rows, K / 2] E2M1 codes
    const uint8_t* as;       // [rows, K / 32] scale bytes
    const int32_t* offsets;  // [G + 1] device
    int G, rows, K, N;
    const uint8_t* w;        // [G, N, K / 2]
    const uint8_t* ws;       // [G, N, K / 32]
    void* out;               // [rows, N] fp32 or bf16
};
hipError_t launch_grouped_gemm_mxfp4(bool f32, const Fp4GemmArgs& g, hipStream_t stream);

}  // namespace moe
