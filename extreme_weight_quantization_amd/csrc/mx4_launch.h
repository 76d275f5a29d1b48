// Host-side launchers of the MX4 operators (called by the C ABI in mx4_api.hip and moe_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act_launch.h"

namespace aqlm {

// fp16 [blocks][32] to codes [blocks][16] and scales [blocks], and back (mx4_convert.hip).
hipError_t launch_mx4_quantize(const void* w, void* codes, void* scales, int64_t blocks, hipStream_t stream);
hipError_t launch_mx4_decode(const void* codes, const void* scales, void* w, int64_t blocks, hipStream_t stream);

// Activations of an MX4 product: fp16 rows (scales NULL), or MX4 codes and scales.
struct MxInput {
    const void* x;
    const void* scales;
};

// Bytes of workspace launch_mx4_linear needs (fp32 parts), for any batch up to `batch`.
int64_t mx4_linear_workspace(bool x_mx4, int64_t out, int64_t in, int64_t batch);
// y = act(W x + bias) + residual (Epilogue's first entries).
hipError_t launch_mx4_linear(const void* codes, const void* scales, MxInput x, const Epilogue& e, void* workspace,
                             int64_t out, int64_t in, int64_t batch, hipStream_t stream);

}  // namespace aqlm
