// C ABI of the MX4 operators (declared in include/aqlm.h): argument checks on the host, then the launches on the caller's
// stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/aqlm.h"
#include "aqlm_validate.h"
#include "mx4_launch.h"

namespace aqlm {

namespace {

constexpr int64_t kMxMaxRows = (int64_t)1 << 40;   // quantize, decode: blocks and addresses stay in 64 bits

bool in_ok(int64_t in) { return in >= 32 && in <= AQLM_MAX_IN && in % 32 == 0; }

int check_linear(int act, int64_t out, int64_t in, int64_t batch) {
    if (act < AQLM_ACT_NONE || act > AQLM_ACT_GELU_TANH) return AQLM_ERR_ACT;
    if (!in_ok(in) || out < 0 || out > AQLM_ACT_MAX_OUT || batch < 0 || batch > AQLM_MX4_MAX_BATCH) return AQLM_ERR_SHAPE;
    // output tiles are counted in 32 bits
    if (((out + 127) / 128 + 1) * ((batch + 127) / 128 + 1) > INT32_MAX) return AQLM_ERR_SHAPE;
    return AQLM_OK;
}

}  // namespace

}  // namespace aqlm

using namespace aqlm;

extern "C" {

int aqlm_mx4_quantize(const void* w, void* codes, void* scales, int64_t rows, int64_t in, void* stream) {
    if (!in_ok(in) || rows < 0 || rows > kMxMaxRows) return AQLM_ERR_SHAPE;
    if (rows == 0) return AQLM_OK;
    if (!w || !codes || !scales) return AQLM_ERR_NULL;
    if (!aligned(w, 16) || !aligned(codes, 16)) return AQLM_ERR_ALIGN;
    return finish(launch_mx4_quantize(w, codes, scales, rows * (in / 32), (hipStream_t)stream));
}

int aqlm_mx4_decode(const void* codes, const void* scales, void* w, int64_t rows, int64_t in, void* stream) {
    if (!in_ok(in) || rows < 0 || rows > kMxMaxRows) return AQLM_ERR_SHAPE;
    if (rows == 0) return AQLM_OK;
    if (!w || !codes || !scales) return AQLM_ERR_NULL;
    if (!aligned(w, 16) || !aligned(codes, 16)) return AQLM_ERR_ALIGN;
    return finish(launch_mx4_decode(codes, scales, w, rows * (in / 32), (hipStream_t)stream));
}

int aqlm_mx4_linear_workspace_bytes(int x_mx4, int64_t out, int64_t in, int64_t batch, int64_t* bytes) {
    if (!bytes) return AQLM_ERR_NULL;
    const int st = check_linear(AQLM_ACT_NONE, out, in, batch);
    if (st != AQLM_OK) return st;
    *bytes = mx4_linear_workspace(x_mx4 != 0, out, in, batch);
    return AQLM_OK;
}

int aqlm_mx4_linear(const void* codes, const void* scales, const void* x, const void* x_scales, const void* bias,
                    const void* residual, void* y, void* workspace, int64_t workspace_bytes, int act, int64_t out,
                    int64_t in, int64_t batch, void* stream) {
    const int st = check_linear(act, out, in, batch);
    if (st != AQLM_OK) return st;
    if (out == 0 || batch == 0) return AQLM_OK;
    if (!codes || !scales || !x || !y) return AQLM_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(bias, 2))
        return AQLM_ERR_ALIGN;
    const int64_t need = mx4_linear_workspace(x_scales != nullptr, out, in, batch);
    if (need > 0) {
        if (!workspace) return AQLM_ERR_NULL;
        if (!aligned(workspace, 16)) return AQLM_ERR_ALIGN;
        if (workspace_bytes < need) return AQLM_ERR_SHAPE;
    }
    Epilogue e = {};
    e.bias[0] = bias;
    e.residual = residual;
    e.y = y;
    e.act = act;
    return finish(launch_mx4_linear(codes, scales, MxInput{x, x_scales}, e, workspace, out, in, batch, (hipStream_t)stream));
}

}  // extern "C"
