// Internal launch interface between the operators' entry points
// (moe_ops.hip) and their kernels.  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace ops {

// Product of e4m3 rows, grouped by expert, with e4m3 weights.
struct ExpertProduct {
    int64_t rows;             // room of x and the output; offsets are held to it
    int E;
    int n;                    // weight rows per expert: N, or 2F (gate, then up)
    int k;
    const uint8_t* x;         // [rows][k]
    const float* xs;          // [rows][k/128]
    const int32_t* offsets;   // [E+1]
    const uint8_t* w;         // [E][n][k]
    const float* ws;          // [E][ceil(n/128)][k/128]
    uint16_t* y;              // product: bf16 [rows][n]
    uint8_t* h;               // gate_up: e4m3 [rows][F]
    float* hs;                //          fp32 [rows][F/128]
};

hipError_t launch_expert_matmul(const ExpertProduct& p, hipStream_t stream);
hipError_t launch_expert_gate_up(const ExpertProduct& p, hipStream_t stream);
// The form that a call of these rows, E and n takes, for the tests.
const char* product_form(bool gate_up, const ExpertProduct& p);

hipError_t launch_add_rmsnorm(int64_t rows, int hidden, const uint16_t* x, const uint16_t* residual,
                              const uint16_t* weight, float eps, uint16_t* residual_out, uint16_t* y,
                              uint8_t* yq, float* ys, hipStream_t stream);

hipError_t launch_topk_route(int64_t tokens, int E, int K, const void* logits, int bf16, int renorm,
                             int32_t* idx, float* w, hipStream_t stream);

struct FewTokens {
    int T, E, K, H, F;
    const uint16_t* x;        // bf16 [T][H]
    const int32_t* idx;       // [T][K]
    const float* w;           // [T][K]
    const uint8_t* w13;       // [E][2F][H]
    const float* s13;         // [E][2F/128][H/128]
    const uint8_t* w2;        // [E][H][F]
    const float* s2;          // [E][H/128][F/128]
    uint16_t* out;            // bf16 [T][H]
    void* workspace;
};

size_t few_token_workspace(int T, int K, int H, int F);
// The form that a call of these sizes takes, for the tests.
const char* few_token_form(const FewTokens& p);
hipError_t launch_few_token_layer(const FewTokens& p, hipStream_t stream);

}  // namespace ops
}  // namespace moe
