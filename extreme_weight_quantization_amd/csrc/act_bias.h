// The second half of the bias gradients: the sums of act_grad_kernel's chunks of tokens.
#pragma once
#include "aqlm_device.h"

namespace aqlm {

struct BiasSum {
    const float* partial;   // [chunk][layer][out]; NULL: nothing to do
    f16* dbias[2];
    int n, out, chunks;
};
constexpr int kBiasSumCols = 64;   // sums a workgroup of 256 threads
inline int64_t bias_sum_blocks(const BiasSum& b) {
    return b.partial == nullptr ? 0 : ((int64_t)b.n * b.out + kBiasSumCols - 1) / kBiasSumCols;
}

// Block blk: wave w adds the w-th of four runs of the chunks, eight loads in flight, then the runs
// are added in order.
__device__ __forceinline__ void bias_sum_block(const BiasSum& b, int64_t blk) {
    __shared__ float red[4][kBiasSumCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i = blk * kBiasSumCols + lane, per = (int64_t)b.n * b.out;
    const int run = (b.chunks + 3) / 4, c1 = min(b.chunks, (wave + 1) * run);
    float s = 0.f;
    for (int c = wave * run; c < c1; c += 8) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = i < per && c + q < c1 ? b.partial[(size_t)(c + q) * per + i] : 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += v[q];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || i >= per) return;
    s = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
    if (i < b.out) b.dbias[0][i] = (f16)s;
    else b.dbias[1][i - b.out] = (f16)s;
}

}  // namespace aqlm
