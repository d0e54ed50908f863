// C ABI of the mixture-of-experts layer for a few tokens (declared in
// include/tgemm.h).  Host code only.
#include <hip/hip_runtime.h>

#include <new>

#include "capi_util.hpp"

using tg::capi_aligned;
using tg::capi_fail;
using tg::capi_ok;
using tg::capi_overlap;

struct gemm_group_mlp_plan {
    gemm_group_mlp_plan_info info;
    gemm_group_plan *up, *down;      // the experts' matrices: their checks and their pre-shuffled images
    int act, slots;
};

namespace {

constexpr int64_t kRange = (int64_t)1 << 31;     // bytes one buffer resource of the kernels covers

size_t pad(size_t n) { return (n + 255) / 256 * 256; }
size_t h_bytes(const gemm_group_mlp_plan *p) { return pad((size_t)p->slots * (size_t)p->info.N * 2); }
size_t y_bytes(const gemm_group_mlp_plan *p) { return pad((size_t)p->slots * (size_t)p->info.K * 4); }

}  // namespace

extern "C" {

gemm_group_mlp_plan *gemm_group_mlp_plan_create(int groups, int64_t tokens, int topk, int64_t K, int64_t N,
                                                int weight_type, int layout, int gated, int epilogue)
{
    if (groups < 1 || groups > GEMM_GROUP_MAX) {
        capi_fail(GEMM_ERR_INVALID_ARG, "groups=%d outside 1..%d", groups, GEMM_GROUP_MAX);
        return nullptr;
    }
    if (tokens < 0 || topk < 1) {
        capi_fail(GEMM_ERR_INVALID_ARG, "tokens=%lld is negative or topk=%d below 1", (long long)tokens, topk);
        return nullptr;
    }
    if (weight_type != GEMM_TYPE_BF16 && weight_type != GEMM_TYPE_E4M3) {
        if (weight_type == GEMM_TYPE_F32)
            capi_fail(GEMM_ERR_UNSUPPORTED, "the layer's weights are bf16 or e4m3");
        else
            capi_fail(GEMM_ERR_INVALID_ARG, "unknown weight_type %d", weight_type);
        return nullptr;
    }
    if (layout < GEMM_LAYOUT_BT || layout > GEMM_LAYOUT_AT_BN) {
        capi_fail(GEMM_ERR_INVALID_ARG, "unknown layout %d", layout);
        return nullptr;
    }
    if (layout != GEMM_LAYOUT_BT && layout != GEMM_LAYOUT_BT_PRESHUFFLED) {
        capi_fail(GEMM_ERR_UNSUPPORTED, "the layer's weights are GEMM_LAYOUT_BT or GEMM_LAYOUT_BT_PRESHUFFLED");
        return nullptr;
    }
    if (gated != 0 && gated != 1) {
        capi_fail(GEMM_ERR_INVALID_ARG, "gated=%d is neither 0 nor 1", gated);
        return nullptr;
    }
    if (epilogue < GEMM_EPI_NONE || epilogue > GEMM_EPI_BIAS_GELU) {
        capi_fail(GEMM_ERR_INVALID_ARG, "unknown epilogue %d", epilogue);
        return nullptr;
    }
    if (tokens > GEMM_GROUP_MLP_MAX_TOKENS || topk > GEMM_GROUP_MLP_MAX_TOPK) {
        capi_fail(GEMM_ERR_UNSUPPORTED,
                  "tokens=%lld above %d or topk=%d above %d (gemm_group_run's products have no such limit%s%s)",
                  (long long)tokens, GEMM_GROUP_MLP_MAX_TOKENS, topk, GEMM_GROUP_MLP_MAX_TOPK,
                  gated ? ", but do not multiply by the gate" : "",
                  weight_type == GEMM_TYPE_E4M3 ? ", but take e4m3 rows beside e4m3 weights" : "");
        return nullptr;
    }
    if (K < 1 || N < 1) {
        capi_fail(GEMM_ERR_INVALID_ARG, "K=%lld and N=%lld must be positive", (long long)K, (long long)N);
        return nullptr;
    }
    if (K > ((int64_t)1 << 20) || N > ((int64_t)1 << 20)) {
        capi_fail(GEMM_ERR_UNSUPPORTED, "K or N above 2^20");
        return nullptr;
    }
    const int64_t slots = tokens * topk;
    if (slots * N * 2 >= kRange) {
        capi_fail(GEMM_ERR_UNSUPPORTED, "tokens x topk x N must stay below 2^30 (32-bit offsets)");
        return nullptr;
    }
    const int dtype = weight_type == GEMM_TYPE_E4M3 ? GEMM_E4M3_OUT_BF16 : GEMM_BF16_OUT_BF16;
    gemm_group_mlp_plan *p = new (std::nothrow) gemm_group_mlp_plan();
    if (!p) {
        capi_fail(GEMM_ERR_INVALID_ARG, "out of host memory");
        return nullptr;
    }
    // The products' own checks; rows of whole 64 bytes make K and N multiples
    // of 32 (e4m3: 64), so every column tile is whole.
    p->up = gemm_group_plan_create(groups, 1, gated ? 2 * N : N, K, dtype, layout);
    p->down = p->up ? gemm_group_plan_create(groups, 1, K, N, dtype, layout) : nullptr;
    if (!p->down) {
        gemm_group_plan_destroy(p->up);
        delete p;
        return nullptr;                  // the message is the product's
    }
    static const int kAct[] = {tg::kActNone, tg::kActNone, tg::kActRelu, tg::kActSilu, tg::kActGelu};
    p->act = kAct[epilogue];
    p->slots = (int)slots;
    gemm_group_mlp_plan_info &I = p->info;
    I.tokens = tokens;
    I.K = K;
    I.N = N;
    I.groups = groups;
    I.topk = topk;
    I.weight_type = weight_type;
    I.layout = layout;
    I.gated = gated;
    I.epilogue = epilogue;
    capi_ok();
    return p;
}

void gemm_group_mlp_plan_destroy(gemm_group_mlp_plan *plan)
{
    if (plan) {
        gemm_group_plan_destroy(plan->up);
        gemm_group_plan_destroy(plan->down);
    }
    delete plan;
}

int gemm_group_mlp_plan_query(const gemm_group_mlp_plan *plan, gemm_group_mlp_plan_info *info)
{
    if (!plan || !info)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL plan or info");
    *info = plan->info;
    return capi_ok();
}

size_t gemm_group_mlp_workspace_bytes(const gemm_group_mlp_plan *plan)
{
    if (!plan || plan->slots == 0)
        return 0;
    return h_bytes(plan) + y_bytes(plan) + (size_t)plan->info.K / 32 * 4;
}

int gemm_group_mlp_preshuffle(const gemm_group_mlp_plan *plan, const void *up, void *up_image, const void *down,
                              void *down_image, hipStream_t stream)
{
    if (!plan)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL plan");
    // Both matrices' checks come before the first launch.
    if (!up || !up_image || !down || !down_image)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL up, up_image, down or down_image");
    if (!capi_aligned(up, 16) || !capi_aligned(up_image, 16) || !capi_aligned(down, 16) || !capi_aligned(down_image, 16))
        return capi_fail(GEMM_ERR_INVALID_ARG, "up, down and their images must be 16-byte aligned");
    const size_t ub = gemm_group_preshuffled_b_bytes(plan->up), db = gemm_group_preshuffled_b_bytes(plan->down);
    if (capi_overlap(up_image, ub, up, ub) || capi_overlap(up_image, ub, down, db) ||
        capi_overlap(down_image, db, up, ub) || capi_overlap(down_image, db, down, db) ||
        capi_overlap(up_image, ub, down_image, db))
        return capi_fail(GEMM_ERR_INVALID_ARG, "an image overlaps a matrix or the other image");
    if (int rc = gemm_group_preshuffle_b(plan->up, up, up_image, stream))
        return rc;
    return gemm_group_preshuffle_b(plan->down, down, down_image, stream);
}

int gemm_group_mlp_run(const gemm_group_mlp_plan *plan, const void *x, const int32_t *ids, const float *weights,
                       const gemm_group_mlp_weights *mats, const void *residual, void *out, void *workspace,
                       size_t workspace_bytes, hipStream_t stream)
{
    if (!plan)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL plan");
    const gemm_group_mlp_plan_info &I = plan->info;
    if (I.tokens == 0)
        return capi_ok();
    if (!x || !ids || !mats || !mats->up || !mats->down || !out)
        return capi_fail(GEMM_ERR_INVALID_ARG, "NULL x, ids, weights' description, up, down or out");
    const bool e4m3 = I.weight_type == GEMM_TYPE_E4M3;
    const size_t eb = e4m3 ? 1 : 2, inner = (size_t)I.N * (I.gated ? 2 : 1), G = (size_t)I.groups;
    const size_t xb = (size_t)I.tokens * I.K * 2, tb = (size_t)plan->slots * 4;
    const size_t need = gemm_group_mlp_workspace_bytes(plan);
    if (!workspace || workspace_bytes < need)
        return capi_fail(GEMM_ERR_INVALID_ARG, "the layer needs a workspace of %zu bytes", need);
    if (!capi_aligned(x, 16) || !capi_aligned(mats->up, 16) || !capi_aligned(mats->down, 16) ||
        !capi_aligned(residual, 16) || !capi_aligned(out, 16) || !capi_aligned(workspace, 16))
        return capi_fail(GEMM_ERR_INVALID_ARG,
                         "x, up, down, residual, out and the workspace must be 16-byte aligned");
    const struct {
        const void *p;
        size_t n;
    } in[] = {{x, xb},
              {ids, tb},
              {weights, tb},
              {mats->up, G * inner * (size_t)I.K * eb},
              {mats->down, G * (size_t)I.N * (size_t)I.K * eb},
              {mats->up_scale, G * inner * 4},
              {mats->up_bias, G * inner * 4},
              {mats->down_scale, G * (size_t)I.K * 4},
              {mats->down_bias, G * (size_t)I.K * 4}};
    for (const auto &v : in) {
        if (!capi_aligned(v.p, 4))
            return capi_fail(GEMM_ERR_INVALID_ARG, "ids, weights, scales and biases must be 4-byte aligned");
        if (capi_overlap(out, xb, v.p, v.n) || capi_overlap(workspace, need, v.p, v.n))
            return capi_fail(GEMM_ERR_INVALID_ARG, "out or the workspace overlaps an input");
    }
    if (capi_overlap(workspace, need, out, xb) || capi_overlap(workspace, need, residual, xb) ||
        (residual != out && capi_overlap(residual, xb, out, xb)))
        return capi_fail(GEMM_ERR_INVALID_ARG, "the workspace, out and (other than in place) the residual overlap");
    if (int rc = tg::capi_check_device())
        return rc;
    tg::MlpArgs a{};
    a.x = x;
    a.ids = ids;
    a.weights = weights;
    a.up = mats->up;
    a.down = mats->down;
    a.up_scale = mats->up_scale;
    a.down_scale = mats->down_scale;
    a.up_bias = mats->up_bias;
    a.down_bias = mats->down_bias;
    a.residual = residual;
    a.out = out;
    a.h = workspace;
    a.y = (float *)((uint8_t *)workspace + h_bytes(plan));
    a.done = (int32_t *)((uint8_t *)workspace + h_bytes(plan) + y_bytes(plan));
    a.groups = I.groups;
    a.tokens = (int32_t)I.tokens;
    a.topk = I.topk;
    a.slots = plan->slots;
    a.K = (int32_t)I.K;
    a.N = (int32_t)I.N;
    a.parts = I.groups < plan->slots ? I.groups : plan->slots;
    a.act = plan->act;
    a.gated = I.gated != 0;
    a.e4m3 = e4m3;
    a.preshuffled = I.layout == GEMM_LAYOUT_BT_PRESHUFFLED;
    const hipError_t e = tg::launch_mlp(a, stream);
    if (e != hipSuccess)
        return capi_fail(GEMM_ERR_HIP, "layer launch: %s", hipGetErrorString(e));
    return capi_ok();
}

}  // extern "C"

static_assert(GEMM_GROUP_MLP_MAX_TOKENS == tg::kMlpTokens && GEMM_GROUP_MLP_MAX_TOPK == tg::kMlpTopk,
              "the header's limits are the kernels'");
