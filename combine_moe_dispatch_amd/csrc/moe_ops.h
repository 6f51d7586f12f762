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

// Tokens sorted by expert and back (sort_rows.hip).
struct SortRows {
    int64_t tokens, rows;
    int K, hidden;
    const void* x;            // sort: tokens' rows; unsort and its gradient: the experts' rows
    const float* xs;          // scales of e4m3 rows, fp32 [tokens][hidden/128]
    const int32_t* slot;      // [tokens][K]
    const float* w;           // [tokens][K] or null: 1
    void* out;
    float* outs;
    const void* dout;         // gradient of the unsorted rows
    void* dy;
    float* dw;
};

size_t sort_workspace(int64_t pairs, int E);
hipError_t launch_sort_plan(int64_t pairs, int E, const int32_t* idx, int32_t* offsets, int32_t* slot,
                            int32_t* source, void* workspace, hipStream_t stream);
hipError_t launch_sort_rows(const SortRows& p, int elem_bytes, hipStream_t stream);
hipError_t launch_unsort_rows(const SortRows& p, bool f32, hipStream_t stream);
hipError_t launch_unsort_rows_grad(const SortRows& p, bool f32, hipStream_t stream);

struct RouteGrad {
    int64_t tokens;
    int E, K;
    const void* logits;
    int bf16, renorm, out_bf16;
    const int32_t* idx;       // [tokens][K]
    const float* dw;          // [tokens][K]
    void* dlogits;
};

hipError_t launch_topk_route_grad(const RouteGrad& a, hipStream_t stream);

// The bf16 product of rows grouped by expert, and its gradients
// (expert_linear.hip).
struct Linear {
    int64_t rows;
    int E, n, k;
    const int32_t* offsets;   // [E+1], null: all rows belong to the one expert
    const uint16_t* x;        // [rows][k] (forward, gradient of the weights)
    const uint16_t* dz;       // [rows][n] (gradients)
    const uint16_t* w;        // [E][n][k]
    const uint16_t* bias;     // [E][n] or null
    int act;                  // moe_activation
    const uint16_t* residual; // or null
    const uint16_t* z_in;     // gradients: pre-activations
    uint16_t* z_out;          // forward: pre-activations, or null
    void* out;                // rows, or the weights' gradient
    int out_f32;
    float* dbias;             // [E][n] or null
    void* workspace;
};

// The tile and splits that a call takes (kind 0 the product, 1 the gradient to
// its input, 2 to its weights, 3 in fp32), for the tests.
const char* linear_form(int kind, bool gated, int64_t rows, int E, int n, int k, int* splits);
size_t linear_workspace(int64_t rows, int E, int n, int k);
hipError_t launch_linear(const Linear& p, hipStream_t stream);
hipError_t launch_linear_grad_input(const Linear& p, hipStream_t stream);
hipError_t launch_linear_grad_weight(const Linear& p, hipStream_t stream);
hipError_t launch_activation_grad(const Linear& p, const uint16_t* dy, hipStream_t stream);

}  // namespace ops
}  // namespace moe
