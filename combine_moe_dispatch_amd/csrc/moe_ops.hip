// Entry points of the operators around dispatch and combine and of the expert
// layer on one card (include/moe_ep.h, under these headings): argument validation
// and launches on the caller's stream.
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

bool has_space(const void* workspace, size_t bytes, size_t needed)
{
    return fine(workspace) && bytes >= needed && (needed == 0 || workspace);
}

bool sort_sizes(int32_t tokens, int32_t E, int32_t top_k)
{
    return tokens >= 0 && E >= 1 && E <= moe::MAX_EXPERTS && top_k >= 1 && top_k <= moe::MAX_TOPK &&
           (int64_t)tokens * top_k <= INT32_MAX;
}

bool row_sizes(int32_t tokens, int32_t top_k, int32_t rows, int32_t hidden)
{
    return tokens >= 0 && top_k >= 1 && top_k <= moe::MAX_TOPK && rows >= 0 && hidden >= 8 &&
           hidden <= MAX_WIDTH && hidden % 8 == 0;
}

bool linear_sizes(int32_t rows, int32_t E, int32_t n, int32_t k)
{
    return rows >= 0 && E >= 1 && E <= moe::MAX_EXPERTS && n >= 8 && n <= MAX_WIDTH && n % 8 == 0 && k >= 8 &&
           k <= MAX_WIDTH && k % 8 == 0;
}

bool offsets_ok(int32_t E, const int32_t* offsets) { return offsets ? aligned16(offsets) : E == 1; }

bool known_activation(int32_t a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_SWIGLU; }

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

// These three are not part of the public ABI: which kernels a call takes (n: weight
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

const char* moe_ops_linear_form(int32_t kind, int32_t gated, int32_t rows, int32_t num_experts, int32_t n, int32_t k,
                                int32_t* splits)
{
    if (kind < 0 || kind > 3 || !linear_sizes(rows, num_experts, n, k) || (gated && (kind != 0 || n % 16 != 0)))
        return "";
    return moe::ops::linear_form(kind, gated != 0, rows, num_experts, n, k, splits);
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

size_t moe_sort_workspace(int32_t tokens, int32_t num_experts, int32_t top_k)
{
    if (!sort_sizes(tokens, num_experts, top_k))
        return 0;
    return moe::ops::sort_workspace((int64_t)tokens * top_k, num_experts);
}

int moe_sort_plan(int32_t tokens, int32_t num_experts, int32_t top_k, const int32_t* topk_idx,
                  int32_t* expert_offsets, int32_t* slot, int32_t* source, void* workspace,
                  size_t workspace_bytes, hipStream_t stream)
{
    CallRange range("moe_sort_plan");
    if (!sort_sizes(tokens, num_experts, top_k))
        return MOE_ERR_INVALID;
    if (!good(expert_offsets) || !fine(source) || !fine(workspace))
        return MOE_ERR_INVALID;
    if (tokens > 0 && (!good(topk_idx) || !good(slot)))
        return MOE_ERR_INVALID;
    const int64_t pairs = (int64_t)tokens * top_k;
    if (!has_space(workspace, workspace_bytes, moe::ops::sort_workspace(pairs, num_experts)))
        return MOE_ERR_INVALID;
    return from_hip(moe::ops::launch_sort_plan(pairs, num_experts, topk_idx, expert_offsets, slot, source,
                                               workspace, stream));
}

int moe_sort_rows(int32_t tokens, int32_t top_k, int32_t rows, int32_t hidden, int32_t dtype, const void* x,
                  const float* x_scale, const int32_t* slot, void* sorted, float* sorted_scale,
                  hipStream_t stream)
{
    CallRange range("moe_sort_rows");
    const bool coded = dtype == MOE_FP8_E4M3;
    if (!row_sizes(tokens, top_k, rows, hidden) || (!coded && dtype != MOE_BF16 && dtype != MOE_FP32))
        return MOE_ERR_INVALID;
    if (coded ? hidden % 128 != 0 : x_scale || sorted_scale)
        return MOE_ERR_INVALID;
    if (tokens == 0)
        return MOE_OK;
    if (!good(x) || !good(slot) || (rows > 0 && !good(sorted)))
        return MOE_ERR_INVALID;
    if (coded && (!good(x_scale) || (rows > 0 && !good(sorted_scale))))
        return MOE_ERR_INVALID;
    moe::ops::SortRows p{};
    p.tokens = tokens;
    p.rows = rows;
    p.K = top_k;
    p.hidden = hidden;
    p.x = x;
    p.xs = x_scale;
    p.slot = slot;
    p.out = sorted;
    p.outs = sorted_scale;
    return from_hip(moe::ops::launch_sort_rows(p, coded ? 1 : dtype == MOE_BF16 ? 2 : 4, stream));
}

int moe_unsort_rows(int32_t tokens, int32_t top_k, int32_t rows, int32_t hidden, int32_t dtype, const void* y,
                    const int32_t* slot, const float* topk_weights, void* out, hipStream_t stream)
{
    CallRange range("moe_unsort_rows");
    if (!row_sizes(tokens, top_k, rows, hidden) || (dtype != MOE_BF16 && dtype != MOE_FP32))
        return MOE_ERR_INVALID;
    if (tokens == 0)
        return MOE_OK;
    if ((rows > 0 && !good(y)) || !good(slot) || !fine(topk_weights) || !good(out))
        return MOE_ERR_INVALID;
    moe::ops::SortRows p{};
    p.tokens = tokens;
    p.rows = rows;
    p.K = top_k;
    p.hidden = hidden;
    p.x = y;
    p.slot = slot;
    p.w = topk_weights;
    p.out = out;
    return from_hip(moe::ops::launch_unsort_rows(p, dtype == MOE_FP32, stream));
}

int moe_unsort_rows_grad(int32_t tokens, int32_t top_k, int32_t rows, int32_t hidden, int32_t dtype,
                         const void* dout, const void* y, const int32_t* slot, const float* topk_weights,
                         void* dy, float* dweights, hipStream_t stream)
{
    CallRange range("moe_unsort_rows_grad");
    if (!row_sizes(tokens, top_k, rows, hidden) || (dtype != MOE_BF16 && dtype != MOE_FP32))
        return MOE_ERR_INVALID;
    if (tokens == 0)
        return MOE_OK;
    if (rows > 0 && ((!dy && !dweights) || !fine(dy) || !fine(y) || (dweights && !y)))
        return MOE_ERR_INVALID;
    if (!good(dout) || !good(slot) || !fine(topk_weights) || !fine(dweights))
        return MOE_ERR_INVALID;
    moe::ops::SortRows p{};
    p.tokens = tokens;
    p.rows = rows;
    p.K = top_k;
    p.hidden = hidden;
    p.x = y;
    p.slot = slot;
    p.w = topk_weights;
    p.dout = dout;
    p.dy = dy;
    p.dw = dweights;
    return from_hip(moe::ops::launch_unsort_rows_grad(p, dtype == MOE_FP32, stream));
}

int moe_topk_route_grad(int32_t tokens, int32_t num_experts, int32_t top_k, const void* logits,
                        int32_t logits_dtype, int32_t renormalise, const int32_t* topk_idx,
                        const float* dweights, void* dlogits, int32_t dlogits_dtype, hipStream_t stream)
{
    CallRange range("moe_topk_route_grad");
    if (tokens < 0 || num_experts < 1 || num_experts > moe::MAX_EXPERTS || top_k < 1 ||
        top_k > moe::MAX_TOPK || top_k > num_experts)
        return MOE_ERR_INVALID;
    if ((logits_dtype != MOE_BF16 && logits_dtype != MOE_FP32) ||
        (dlogits_dtype != MOE_BF16 && dlogits_dtype != MOE_FP32))
        return MOE_ERR_INVALID;
    if (tokens == 0)
        return MOE_OK;
    if (!good(logits) || !good(topk_idx) || !good(dweights) || !good(dlogits))
        return MOE_ERR_INVALID;
    moe::ops::RouteGrad a{};
    a.tokens = tokens;
    a.E = num_experts;
    a.K = top_k;
    a.logits = logits;
    a.bf16 = logits_dtype == MOE_BF16;
    a.renorm = renormalise != 0;
    a.out_bf16 = dlogits_dtype == MOE_BF16;
    a.idx = topk_idx;
    a.dw = dweights;
    a.dlogits = dlogits;
    return from_hip(moe::ops::launch_topk_route_grad(a, stream));
}

size_t moe_expert_linear_workspace(int32_t rows, int32_t num_experts, int32_t n, int32_t k)
{
    return linear_sizes(rows, num_experts, n, k) ? moe::ops::linear_workspace(rows, num_experts, n, k) : 0;
}

int moe_expert_linear(int32_t rows, int32_t num_experts, int32_t n, int32_t k, const void* x,
                      const int32_t* expert_offsets, const void* w, const void* bias, int32_t activation,
                      const void* residual, void* z, void* y, int32_t y_dtype, void* workspace,
                      size_t workspace_bytes, hipStream_t stream)
{
    CallRange range("moe_expert_linear");
    if (!linear_sizes(rows, num_experts, n, k) || !known_activation(activation) ||
        (activation == MOE_ACT_SWIGLU && n % 16 != 0) || (y_dtype != MOE_BF16 && y_dtype != MOE_FP32))
        return MOE_ERR_INVALID;
    if (rows == 0)
        return MOE_OK;
    if (!good(x) || !offsets_ok(num_experts, expert_offsets) || !good(w) || !fine(bias) || !fine(residual) ||
        !fine(z) || !good(y) || (y_dtype == MOE_FP32 && residual == y) ||
        !has_space(workspace, workspace_bytes, moe::ops::linear_workspace(rows, num_experts, n, k)))
        return MOE_ERR_INVALID;
    moe::ops::Linear p{};
    p.rows = rows;
    p.E = num_experts;
    p.n = n;
    p.k = k;
    p.offsets = expert_offsets;
    p.x = (const uint16_t*)x;
    p.w = (const uint16_t*)w;
    p.bias = (const uint16_t*)bias;
    p.act = activation;
    p.residual = (const uint16_t*)residual;
    p.z_out = (uint16_t*)z;
    p.out = y;
    p.out_f32 = y_dtype == MOE_FP32;
    p.workspace = workspace;
    return from_hip(moe::ops::launch_linear(p, stream));
}

int moe_activation_grad(int32_t rows, int32_t num_experts, int32_t n, int32_t activation,
                        const int32_t* expert_offsets, const void* z, const void* dy, void* dz,
                        hipStream_t stream)
{
    CallRange range("moe_activation_grad");
    if (!linear_sizes(rows, num_experts, n, 8) || !known_activation(activation) || activation == MOE_ACT_NONE ||
        (activation == MOE_ACT_SWIGLU && (n % 16 != 0 || (dy && dz == dy))))
        return MOE_ERR_INVALID;
    if (rows == 0)
        return MOE_OK;
    if (!offsets_ok(num_experts, expert_offsets) || !good(z) || !good(dy) || !good(dz))
        return MOE_ERR_INVALID;
    moe::ops::Linear p{};
    p.rows = rows;
    p.E = num_experts;
    p.n = n;
    p.offsets = expert_offsets;
    p.act = activation;
    p.z_in = (const uint16_t*)z;
    p.out = dz;
    return from_hip(moe::ops::launch_activation_grad(p, (const uint16_t*)dy, stream));
}

int moe_expert_linear_grad_input(int32_t rows, int32_t num_experts, int32_t n, int32_t k, const void* dz,
                                 const int32_t* expert_offsets, const void* w, int32_t activation,
                                 const void* z, const void* residual, void* dx, int32_t dx_dtype,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    CallRange range("moe_expert_linear_grad_input");
    if (!linear_sizes(rows, num_experts, n, k) || !known_activation(activation) ||
        (dx_dtype != MOE_BF16 && dx_dtype != MOE_FP32) || (activation == MOE_ACT_NONE) != (z == nullptr))
        return MOE_ERR_INVALID;
    if (rows == 0)
        return MOE_OK;
    if (!good(dz) || !offsets_ok(num_experts, expert_offsets) || !good(w) || !fine(z) || !fine(residual) ||
        !good(dx) || (dx_dtype == MOE_FP32 && residual == dx) ||
        !has_space(workspace, workspace_bytes, moe::ops::linear_workspace(rows, num_experts, n, k)))
        return MOE_ERR_INVALID;
    moe::ops::Linear p{};
    p.rows = rows;
    p.E = num_experts;
    p.n = n;
    p.k = k;
    p.offsets = expert_offsets;
    p.dz = (const uint16_t*)dz;
    p.w = (const uint16_t*)w;
    p.act = activation;
    p.z_in = (const uint16_t*)z;
    p.residual = (const uint16_t*)residual;
    p.out = dx;
    p.out_f32 = dx_dtype == MOE_FP32;
    p.workspace = workspace;
    return from_hip(moe::ops::launch_linear_grad_input(p, stream));
}

int moe_expert_linear_grad_weight(int32_t rows, int32_t num_experts, int32_t n, int32_t k, const void* dz,
                                  const void* x, const int32_t* expert_offsets, void* dw, int32_t dw_dtype,
                                  float* dbias, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    CallRange range("moe_expert_linear_grad_weight");
    if (!linear_sizes(rows, num_experts, n, k) || (dw_dtype != MOE_BF16 && dw_dtype != MOE_FP32))
        return MOE_ERR_INVALID;
    if (!good(dw) || !fine(dbias) ||
        (rows > 0 && (!good(dz) || !good(x) || !offsets_ok(num_experts, expert_offsets))) ||
        !has_space(workspace, workspace_bytes, moe::ops::linear_workspace(rows, num_experts, n, k)))
        return MOE_ERR_INVALID;
    moe::ops::Linear p{};
    p.rows = rows;
    p.E = num_experts;
    p.n = n;
    p.k = k;
    p.offsets = rows > 0 ? expert_offsets : nullptr;
    p.x = (const uint16_t*)x;
    p.dz = (const uint16_t*)dz;
    p.out = dw;
    p.out_f32 = dw_dtype == MOE_FP32;
    p.dbias = dbias;
    p.workspace = workspace;
    return from_hip(moe::ops::launch_linear_grad_weight(p, stream));
}

}  // extern "C"
