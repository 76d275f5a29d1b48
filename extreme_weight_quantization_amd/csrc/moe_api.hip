// C ABI of the mixture-of-experts operators (declared in include/aqlm.h): argument checks on the host, then the launches on
// the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/aqlm.h"
#include "aqlm_validate.h"
#include "moe_launch.h"

namespace aqlm {

static_assert(kMoeMaxExperts == AQLM_MOE_MAX_EXPERTS && kMoeMaxK == AQLM_MOE_MAX_K && kMoeMaxPairs == AQLM_MOE_MAX_PAIRS,
              "limits");
static_assert((int)kScoreSoftmax == AQLM_SCORE_SOFTMAX && (int)kScoreSigmoid == AQLM_SCORE_SIGMOID, "scores");

namespace {

int check_workspace(const void* workspace, int64_t have, int64_t need) {
    if (need == 0) return AQLM_OK;
    if (!workspace) return AQLM_ERR_NULL;
    if (!aligned(workspace, 16)) return AQLM_ERR_ALIGN;
    return have < need ? AQLM_ERR_SHAPE : AQLM_OK;
}

bool experts_ok(int64_t experts, int64_t k) {
    return experts >= 1 && experts <= AQLM_MOE_MAX_EXPERTS && k >= 1 && k <= AQLM_MOE_MAX_K;
}

int check_route(int64_t experts, int64_t in, int64_t k, int64_t tokens) {
    if (!experts_ok(experts, k) || k > experts) return AQLM_ERR_SHAPE;
    if (in < 8 || in > AQLM_MAX_IN || in % 8 != 0 || tokens < 0 || tokens > AQLM_ROUTE_MAX_TOKENS) return AQLM_ERR_SHAPE;
    return AQLM_OK;
}

// Sizes of a layer whose rows come in units of `in_unit` inputs.
int check_layer(int act, int64_t experts, int64_t k, int64_t in, int64_t inner, int64_t tokens, int64_t in_unit) {
    if (act < AQLM_ACT_NONE || act > AQLM_ACT_GELU_TANH) return AQLM_ERR_ACT;
    if (!experts_ok(experts, k) || tokens < 0 || tokens > AQLM_MOE_MAX_PAIRS / k) return AQLM_ERR_SHAPE;
    for (int64_t n : {in, inner})
        if (n < in_unit || n > AQLM_MAX_IN || n % in_unit != 0) return AQLM_ERR_SHAPE;
    return AQLM_OK;
}

int check_call(const MoeCall& c) {
    if (!c.x || !c.ids || !c.weights || !c.y) return AQLM_ERR_NULL;
    if (!aligned(c.x, 16) || !aligned(c.y, 16) || !aligned(c.residual, 16) || !aligned(c.ids, 4) || !aligned(c.weights, 4))
        return AQLM_ERR_ALIGN;
    return AQLM_OK;
}

}  // namespace

}  // namespace aqlm

using namespace aqlm;

extern "C" {

int aqlm_moe_route_workspace_bytes(int64_t experts, int64_t in, int64_t k, int64_t tokens, int64_t* bytes) {
    if (!bytes) return AQLM_ERR_NULL;
    const int st = check_route(experts, in, k, tokens);
    if (st != AQLM_OK) return st;
    *bytes = route_workspace(experts, in, tokens);
    return AQLM_OK;
}

int aqlm_moe_route(const void* x, const void* router, const float* bias, int32_t* ids, float* weights, void* workspace,
                   int64_t workspace_bytes, int score, int renorm, float scale, int64_t experts, int64_t in, int64_t k,
                   int64_t tokens, void* stream) {
    if (score != AQLM_SCORE_SOFTMAX && score != AQLM_SCORE_SIGMOID) return AQLM_ERR_ACT;
    int st = check_route(experts, in, k, tokens);
    if (st != AQLM_OK) return st;
    if (tokens == 0) return AQLM_OK;
    if (!x || !router || !ids || !weights) return AQLM_ERR_NULL;
    if (!aligned(x, 16) || !aligned(router, 16) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return AQLM_ERR_ALIGN;
    st = check_workspace(workspace, workspace_bytes, route_workspace(experts, in, tokens));
    if (st != AQLM_OK) return st;
    const RouteCall c = {x, router, bias, ids, weights, score, renorm != 0, (int)k, (int)experts, scale, in, tokens};
    return finish(launch_route(c, workspace, (hipStream_t)stream));
}

int aqlm_moe_workspace_bytes(int M, int B, int g, int64_t experts, int64_t in, int64_t inner, int64_t k, int64_t tokens,
                             int64_t* bytes) {
    if (!bytes) return AQLM_ERR_NULL;
    if (!generic_scheme_ok(M, B, g)) return AQLM_ERR_SCHEME;
    const int st = check_layer(AQLM_ACT_NONE, experts, k, in, inner, tokens, g);
    if (st != AQLM_OK) return st;
    *bytes = tokens == 0 ? 0 : moe_workspace(in, inner, tokens, k);
    return AQLM_OK;
}

int aqlm_moe(const void* const* codes, const void* const* codebooks, const void* const* scales, const void* x,
             const int32_t* ids, const float* weights, const void* residual, void* y, void* workspace,
             int64_t workspace_bytes, int act, int M, int B, int g, int64_t experts, int64_t in, int64_t inner, int64_t k,
             int64_t tokens, void* stream) {
    if (!generic_scheme_ok(M, B, g)) return AQLM_ERR_SCHEME;
    int st = check_layer(act, experts, k, in, inner, tokens, g);
    if (st != AQLM_OK) return st;
    if (tokens == 0) return AQLM_OK;
    if (!codes || !codebooks || !scales) return AQLM_ERR_NULL;
    MoeLayers L;
    for (int l = 0; l < 3; ++l) {
        if (!codes[l] || !codebooks[l] || !scales[l]) return AQLM_ERR_NULL;
        if (!aligned(codes[l], 16) || !aligned(codebooks[l], 16) || !aligned(scales[l], 2)) return AQLM_ERR_ALIGN;
        L.codes[l] = codes[l];
        L.codebooks[l] = codebooks[l];
        L.scales[l] = scales[l];
    }
    const MoeCall c = {x, ids, weights, residual, y, act, (int)experts, (int)k, (int)tokens, in, inner};
    st = check_call(c);
    if (st != AQLM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, moe_workspace(in, inner, tokens, k));
    if (st != AQLM_OK) return st;
    return finish(launch_moe(GenericScheme{M, B, g}, L, c, workspace, (hipStream_t)stream));
}

int aqlm_moe_mx4_workspace_bytes(int64_t experts, int64_t in, int64_t inner, int64_t k, int64_t tokens, int64_t* bytes) {
    if (!bytes) return AQLM_ERR_NULL;
    const int st = check_layer(AQLM_ACT_NONE, experts, k, in, inner, tokens, 32);
    if (st != AQLM_OK) return st;
    *bytes = tokens == 0 ? 0 : moe_mx4_workspace(in, inner, tokens, k);
    return AQLM_OK;
}

int aqlm_moe_mx4(const void* const* codes, const void* const* scales, const void* x, const int32_t* ids,
                 const float* weights, const void* residual, void* y, void* workspace, int64_t workspace_bytes, int act,
                 int64_t experts, int64_t in, int64_t inner, int64_t k, int64_t tokens, void* stream) {
    int st = check_layer(act, experts, k, in, inner, tokens, 32);
    if (st != AQLM_OK) return st;
    if (tokens == 0) return AQLM_OK;
    if (!codes || !scales) return AQLM_ERR_NULL;
    MoeMx4Layers L;
    for (int l = 0; l < 3; ++l) {
        if (!codes[l] || !scales[l]) return AQLM_ERR_NULL;
        if (!aligned(codes[l], 16)) return AQLM_ERR_ALIGN;
        L.codes[l] = codes[l];
        L.scales[l] = scales[l];
    }
    const MoeCall c = {x, ids, weights, residual, y, act, (int)experts, (int)k, (int)tokens, in, inner};
    st = check_call(c);
    if (st != AQLM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, moe_mx4_workspace(in, inner, tokens, k));
    if (st != AQLM_OK) return st;
    return finish(launch_moe_mx4(L, c, workspace, (hipStream_t)stream));
}

}  // extern "C"
