// Entry points of the operators around dispatch and combine (include/moe_ep.h,
// "Operators around dispatch and combine"): argument validation and launches
// on the caller's stream.
#include "moe_ops.h"

#include <rocprofiler-sdk-roctx/roctx.h>

#include "moe_ep.h"
#include "moe_kernels.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// A ROCTX range around one call, as around the four of moe_ep.hip.
struct CallRange {
    explicit CallRange(const char* name) { roctxRangePushA(name); }
    ~CallRange() { roctxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

constexpr int MAX_WIDTH = 65536;

// A needed device pointer.
bool good(const void* p) { return p && aligned16(p); }
// One that may be absent.
bool fine(const void* p) { return aligned16(p); }

bool width128(int n) { return n >= 128 && n <= MAX_WIDTH && n % 128 == 0; }

// What the two products share.
int check_product(int32_t rows, int32_t E, int32_t k, const void* x, const float* xs,
                  const int32_t* offsets, const void* w, const float* ws)
{
    if (rows < 0 || E < 1 || E > moe::MAX_EXPERTS || !width128(k))
        return MOE_ERR_INVALID;
    if (rows > 0 && (!good(x) || !good(xs) || !good(offsets) || !good(w) || !good(ws)))
        return MOE_ERR_INVALID;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_add_rmsnorm(int32_t rows, int32_t hidden, const void* x, const void* residual, const void* weight,
                    float eps, void* residual_out, void* y, void* y_q, float* y_scale, hipStream_t stream)
{
    CallRange range("moe_add_rmsnorm");
    if (rows < 0 || hidden < 8 || hidden > MAX_WIDTH || hidden % 8 != 0)
        return MOE_ERR_INVALID;
    if (!(eps >= 0.0f) || (!residual_out && !y && !y_q) || (y_q == nullptr) != (y_scale == nullptr))
        return MOE_ERR_INVALID;
    if (y_q && hidden % 128 != 0)
        return MOE_ERR_INVALID;
    if (!fine(residual) || !fine(residual_out) || !fine(y) || !fine(y_q) || !fine(y_scale))
        return MOE_ERR_INVALID;
    if (rows == 0)
        return MOE_OK;
    if (!good(x) || !good(weight))
        return MOE_ERR_INVALID;
    return from_hip(moe::ops::launch_add_rmsnorm(
        rows, hidden, (const uint16_t*)x, (const uint16_t*)residual, (const uint16_t*)weight, eps,
        (uint16_t*)residual_out, (uint16_t*)y, (uint8_t*)y_q, y_scale, stream));
}

int moe_topk_route(int32_t tokens, int32_t num_experts, int32_t top_k, const void* logits,
                   int32_t logits_dtype, int32_t renormalise, int32_t* topk_idx, float* topk_weights,
                   hipStream_t stream)
{
    CallRange range("moe_topk_route");
    if (tokens < 0 || num_experts < 1 || num_experts > moe::MAX_EXPERTS || top_k < 1 ||
        top_k > moe::MAX_TOPK || top_k > num_experts)
        return MOE_ERR_INVALID;
    if (logits_dtype != MOE_BF16 && logits_dtype != MOE_FP32)
        return MOE_ERR_INVALID;
    if (tokens == 0)
        return MOE_OK;
    if (!good(logits) || !good(topk_idx) || !good(topk_weights))
        return MOE_ERR_INVALID;
    return from_hip(moe::ops::launch_topk_route(tokens, num_experts, top_k, logits,
                                                logits_dtype == MOE_BF16, renormalise != 0, topk_idx,
                                                topk_weights, stream));
}

int moe_expert_matmul(int32_t rows, int32_t num_experts, int32_t n, int32_t k, const void* x,
                      const float* x_scale, const int32_t* expert_offsets, const void* w,
                      const float* w_scale, void* y, hipStream_t stream)
{
    CallRange range("moe_expert_matmul");
    const int rc = check_product(rows, num_experts, k, x, x_scale, expert_offsets, w, w_scale);
    if (rc != MOE_OK)
        return rc;
    if (n < 8 || n > MAX_WIDTH || n % 8 != 0)
        return MOE_ERR_INVALID;
    if (rows == 0)
        return MOE_OK;
    if (!good(y))
        return MOE_ERR_INVALID;
    moe::ops::ExpertProduct p{};
    p.rows = rows;
    p.E = num_experts;
    p.n = n;
    p.k = k;
    p.x = (const uint8_t*)x;
    p.xs = x_scale;
    p.offsets = expert_offsets;
    p.w = (const uint8_t*)w;
    p.ws = w_scale;
    p.y = (uint16_t*)y;
    return from_hip(moe::ops::launch_expert_matmul(p, stream));
}

int moe_expert_gate_up(int32_t rows, int32_t num_experts, int32_t f, int32_t k, const void* x,
                       const float* x_scale, const int32_t* expert_offsets, const void* w13,
                       const float* w13_scale, void* h, float* h_scale, hipStream_t stream)
{
    CallRange range("moe_expert_gate_up");
    const int rc = check_product(rows, num_experts, k, x, x_scale, expert_offsets, w13, w13_scale);
    if (rc != MOE_OK)
        return rc;
    if (!width128(f))
        return MOE_ERR_INVALID;
    if (rows == 0)
        return MOE_OK;
    if (!good(h) || !good(h_scale))
        return MOE_ERR_INVALID;
    moe::ops::ExpertProduct p{};
    p.rows = rows;
    p.E = num_experts;
    p.n = 2 * f;
    p.k = k;
    p.x = (const uint8_t*)x;
    p.xs = x_scale;
    p.offsets = expert_offsets;
    p.w = (const uint8_t*)w13;
    p.ws = w13_scale;
    p.h = (uint8_t*)h;
    p.hs = h_scale;
    return from_hip(moe::ops::launch_expert_gate_up(p, stream));
}

// These two are not part of the public ABI: which kernels a call takes (n: weight
// rows per expert, 2f for gate_up), so that tests can say what they check; ""
// for sizes that no call takes.
const char* moe_ops_product_form(int32_t gate_up, int32_t rows, int32_t num_experts, int32_t n)
{
    if (rows < 1 || num_experts < 1 || num_experts > moe::MAX_EXPERTS || n < 8 || n > 2 * MAX_WIDTH)
        return "";
    moe::ops::ExpertProduct p{};
    p.rows = rows;
    p.E = num_experts;
    p.n = n;
    return moe::ops::product_form(gate_up != 0, p);
}

const char* moe_ops_few_token_form(int32_t num_tokens, int32_t num_experts, int32_t top_k, int32_t hidden, int32_t f)
{
    if (num_tokens < 1 || num_tokens > MOE_FEW_TOKENS_MAX || num_experts < 1 || num_experts > moe::MAX_EXPERTS ||
        top_k < 1 || top_k > moe::MAX_TOPK || !width128(hidden) || !width128(f))
        return "";
    moe::ops::FewTokens p{};
    p.T = num_tokens;
    p.E = num_experts;
    p.K = top_k;
    p.H = hidden;
    p.F = f;
    return moe::ops::few_token_form(p);
}

size_t moe_few_token_workspace(int32_t num_tokens, int32_t top_k, int32_t hidden, int32_t f)
{
    if (num_tokens < 1 || num_tokens > MOE_FEW_TOKENS_MAX || top_k < 1 || top_k > moe::MAX_TOPK ||
        !width128(hidden) || !width128(f))
        return 0;
    return moe::ops::few_token_workspace(num_tokens, top_k, hidden, f);
}

int moe_few_token_layer(int32_t num_tokens, int32_t num_experts, int32_t top_k, int32_t hidden, int32_t f,
                        const void* x, const int32_t* topk_idx, const float* topk_weights, const void* w13,
                        const float* w13_scale, const void* w2, const float* w2_scale, void* out,
                        void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    CallRange range("moe_few_token_layer");
    if (num_tokens < 0 || num_tokens > MOE_FEW_TOKENS_MAX || num_experts < 1 ||
        num_experts > moe::MAX_EXPERTS || top_k < 1 || top_k > moe::MAX_TOPK || !width128(hidden) ||
        !width128(f))
        return MOE_ERR_INVALID;
    if (num_tokens == 0)
        return MOE_OK;
    if (!good(x) || !good(topk_idx) || !good(topk_weights) || !good(w13) || !good(w13_scale) || !good(w2) ||
        !good(w2_scale) || !good(out) || !good(workspace))
        return MOE_ERR_INVALID;
    if (workspace_bytes < moe::ops::few_token_workspace(num_tokens, top_k, hidden, f))
        return MOE_ERR_INVALID;
    moe::ops::FewTokens p{};
    p.T = num_tokens;
    p.E = num_experts;
    p.K = top_k;
    p.H = hidden;
    p.F = f;
    p.x = (const uint16_t*)x;
    p.idx = topk_idx;
    p.w = topk_weights;
    p.w13 = (const uint8_t*)w13;
    p.s13 = w13_scale;
    p.w2 = (const uint8_t*)w2;
    p.s2 = w2_scale;
    p.out = (uint16_t*)out;
    p.workspace = workspace;
    return from_hip(moe::ops::launch_few_token_layer(p, stream));
}

}  // extern "C"
