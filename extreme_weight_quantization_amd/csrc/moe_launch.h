// Host-side launchers of the mixture-of-experts operators (called by the C ABI in moe_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act_launch.h"

namespace aqlm {

constexpr int kMoeMaxExperts = 512, kMoeMaxK = 16, kMoeMaxPairs = 1024;

// Router (moe_route.hip).
enum RouteScore : int { kScoreSoftmax = 0, kScoreSigmoid = 1 };
struct RouteCall {
    const void *x, *router;     // fp16 [tokens][in], [experts][in]
    const float* bias;          // [experts] or NULL
    int32_t* ids;               // [tokens][k]
    float* weights;             // [tokens][k]
    int score, renorm, k, experts;
    float scale;
    int64_t in, tokens;
};
int64_t route_workspace(int64_t experts, int64_t in, int64_t tokens);
hipError_t launch_route(const RouteCall& c, void* workspace, hipStream_t stream);

// The layer y_t = residual_t + sum_j w_tj Wd_e (act(Wg_e x_t) * (Wu_e x_t)), e = ids_tj.
struct MoeCall {
    const void* x;              // fp16 [tokens][in]
    const int32_t* ids;         // [tokens][k]
    const float* weights;       // [tokens][k]
    const void* residual;       // fp16 [tokens][in] or NULL; may be y
    void* y;                    // fp16 [tokens][in]
    int act, experts, k, tokens;
    int64_t in, inner;
    int pairs() const { return tokens * k; }
};

// Experts in an AQLM scheme (moe.hip): layers gate, up [experts][inner][in/g][M], down [experts][in][inner/g][M].
struct MoeLayers {
    const void* codes[3];
    const void* codebooks[3];
    const void* scales[3];
};
int64_t moe_workspace(int64_t in, int64_t inner, int64_t tokens, int64_t k);
hipError_t launch_moe(const GenericScheme& sc, const MoeLayers& L, const MoeCall& c, void* workspace, hipStream_t stream);

// Experts in MX4 (moe_mx4.hip): codes gate, up [experts][inner][in/2], down [experts][in][inner/2], scales likewise.
struct MoeMx4Layers {
    const void* codes[3];
    const void* scales[3];
};
int64_t moe_mx4_workspace(int64_t in, int64_t inner, int64_t tokens, int64_t k);
hipError_t launch_moe_mx4(const MoeMx4Layers& L, const MoeCall& c, void* workspace, hipStream_t stream);

// y_t = residual_t + sum over choices j with an expert of w_tj part[t k + j], in the order of j (moe.hip).
hipError_t launch_moe_combine(const float* part, const MoeCall& c, hipStream_t stream);

}  // namespace aqlm
