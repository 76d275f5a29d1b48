// The product of MX4 weights with many tokens (mx4_gemm.hip), as mx4_linear.hip calls it.
#pragma once
#include "mx4.h"
#include "mx4_launch.h"

namespace aqlm {

// Whether it takes this call.
bool mx4_gemm_serves(bool x_mx4, int64_t out, int64_t in, int64_t batch);
// Bytes of fp32 parts it may write for any batch up to this one.
int64_t mx4_gemm_part_bytes(int64_t out, int64_t in, int64_t batch);
// x: MX4, or fp16 rows (scales NULL).
hipError_t launch_mx4_gemm(const void* codes, const void* scales, MxInput x, const Epilogue& e, void* part, int64_t out, int64_t in,
                           int64_t batch, hipStream_t stream);

}  // namespace aqlm
