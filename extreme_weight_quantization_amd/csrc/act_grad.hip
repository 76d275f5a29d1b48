// Gradients of the pre-activations, the first step of the backward passes:
//
//   one layer    dz  = dy act'(z)               (no activation: dz = dy)
//   gated        dzg = dy zu act'(zg),  dzu = dy act(zg)
//   bias         dbias[i] = sum over tokens t of dz[t][i]
//
// computed in fp32 from the fp16 inputs.  dz, times the row's scale where the codewords are
// multiplied as they are, is rounded to fp16 once, in units of a power of two that a token's 512
// columns of a workgroup share (act_math.h): it is the operand of the fp16 matrix cores in dx = dz W.
// The bias sums take the fp32 values, in a fixed
// order: each wave adds its tokens, a workgroup its four waves, and act_bias_kernel the
// workgroups' sums, four runs of them in order and then the runs.
//
// Elementwise, bound by HBM: 2 bytes read per input and element, 2 written.  A thread
// takes 8 consecutive rows of W, 16 bytes of each operand.
#include "act_bias.h"
#include "act_launch.h"
#include "act_math.h"
#include "aqlm_device.h"

namespace aqlm {

namespace {

static_assert(kGradCols == 64 * 8 && kGradCols == kLevelCols, "columns per workgroup: 64 lanes of 8");

struct GradArgs {
    const f16* dy;
    const f16* z[2];
    const f16* scales[2];
    f16* dz;
    int8_t* levels;
    float* partial;
    int out, op, T, n_cols;   // n_cols: workgroups across the columns
};

__device__ __forceinline__ f16x8 load8(const f16* p, int left, bool vec) {
    if (vec) return *reinterpret_cast<const f16x8*>(p);
    f16x8 v;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = q < left ? p[q] : (f16)0.f;
    return v;
}

// The largest of the wave's non-negative values, in a scalar: prefix maxima inside rows of 16 lanes, then
// across them; lane 63 ends up with all.
template <int CTRL>
__device__ __forceinline__ float max_from(float v) {
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = max_from<0x111>(v);   // row_shr 1, 2, 4, 8
    v = max_from<0x112>(v);
    v = max_from<0x114>(v);
    v = max_from<0x118>(v);
    v = max_from<0x142>(v);   // row_bcast 15, 31
    v = max_from<0x143>(v);
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

template <int N, int ACT, int WT>
__global__ __launch_bounds__(256) void act_grad_kernel(GradArgs a) {
    __shared__ float red[3][N][kGradCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cb = (int)(blockIdx.x % a.n_cols), chunk = (int)(blockIdx.x / a.n_cols);
    const int c0 = cb * kGradCols + 8 * lane;
    const int t0 = chunk * 4 * WT, t1 = min(a.T, t0 + 4 * WT);
    const bool vec = a.out % 8 == 0;   // rows of 16-byte chunks
    const int left = a.out - c0;       // columns of this lane inside the matrix
    constexpr int kOps = N == 1 ? 2 : 3;   // dy, then z (gated: zg, zu)
    const int tw = t0 + wave * WT, n_tok = min(WT, t1 - tw);   // may be <= 0
    const bool in_row = left > 0;
    // every load of the wave's tokens first; a token past the batch repeats the last one
    f16x8 v[WT][kOps];
    if (in_row && n_tok > 0) {
#pragma unroll
        for (int i = 0; i < WT; ++i) {
            const size_t at = (size_t)(tw + min(i, n_tok - 1)) * a.out + c0;
            v[i][0] = load8(a.dy + at, left, vec);
            if (N > 1 || ACT != kActNone) v[i][1] = load8(a.z[0] + at, left, vec);
            if constexpr (N > 1) v[i][kOps - 1] = load8(a.z[N - 1] + at, left, vec);
        }
    }
    float m[N][8], sum[N][8];
#pragma unroll
    for (int l = 0; l < N; ++l)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            m[l][q] = (a.scales[l] != nullptr && q < left) ? (float)a.scales[l][c0 + q] : 1.f;
            sum[l][q] = 0.f;
        }
#pragma unroll
    for (int i = 0; i < WT; ++i) {
        if (i >= n_tok) break;
        float g[N][8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float dy = (float)v[i][0][q], z = (float)v[i][1][q];
            if constexpr (N == 1) {
                g[0][q] = ACT == kActNone ? dy : dy * act_slope<ACT>(z);
            } else {
                g[0][q] = dy * (float)v[i][kOps - 1][q] * act_slope<ACT>(z);
                g[N - 1][q] = dy * act_value<ACT>(z);
            }
        }
#pragma unroll
        for (int l = 0; l < N; ++l) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                g[l][q] = q < left ? g[l][q] : 0.f;
                sum[l][q] += g[l][q];
                g[l][q] = q < left ? g[l][q] * m[l][q] : 0.f;
            }
            if (a.dz == nullptr) continue;
            const int level = grad_level(wave_max(largest_finite(g[l])));
            const float unit = level_unit(-level);
            f16x8 o;
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = (f16)(g[l][q] * unit);
            if (c0 < a.op)
                *reinterpret_cast<u32x4*>(a.dz + (size_t)(tw + i) * (N * a.op) + (size_t)l * a.op + c0) = as_u32x4(o);
            if (lane == 0) a.levels[((size_t)(tw + i) * N + l) * a.n_cols + cb] = (int8_t)level;
        }
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int l = 0; l < N; ++l)
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (wave > 0) red[wave - 1][l][8 * lane + q] = sum[l][q];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int l = 0; l < N; ++l)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float s = sum[l][q];
#pragma unroll
            for (int w = 0; w < 3; ++w) s += red[w][l][8 * lane + q];
            if (q < left) a.partial[((size_t)chunk * N + l) * a.out + c0 + q] = s;
        }
}

__global__ __launch_bounds__(256) void act_bias_kernel(const BiasSum b) { bias_sum_block(b, blockIdx.x); }

__global__ __launch_bounds__(256) void zero16_kernel(f16* p, int64_t n) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) p[i] = (f16)0.f;
}

}  // namespace

namespace {

template <int N, int WT>
auto grad_kernel_of(int act) {
    switch (act) {
        case kActRelu: return act_grad_kernel<N, kActRelu, WT>;
        case kActSilu: return act_grad_kernel<N, kActSilu, WT>;
        case kActGelu: return act_grad_kernel<N, kActGelu, WT>;
        case kActGeluTanh: return act_grad_kernel<N, kActGeluTanh, WT>;
        default: return act_grad_kernel<N, kActNone, WT>;
    }
}

auto grad_kernel(int n, int act, int wave_tokens) {
    if (wave_tokens == 1) return n == 1 ? grad_kernel_of<1, 1>(act) : grad_kernel_of<2, 1>(act);
    return n == 1 ? grad_kernel_of<1, 4>(act) : grad_kernel_of<2, 4>(act);
}

}  // namespace

hipError_t launch_zero16(void* p, int64_t n, hipStream_t stream) {
    if (n <= 0) return hipSuccess;
    int64_t blocks = (n + 255) / 256;
    const int64_t cap = (int64_t)device_cu_count() * 16;
    if (blocks > cap) blocks = cap;
    hipLaunchKernelGGL(zero16_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, static_cast<f16*>(p), n);
    return hipGetLastError();
}

int64_t grad_chunks(int64_t out, int64_t batch) {
    const int64_t per = 4 * grad_wave_tokens(out, batch);
    return (batch + per - 1) / per;
}

hipError_t launch_act_grad(const void* dy, const void* const* z, const void* const* scales, int n, int act, void* dz,
                           float* partial, int64_t out, int64_t op, int64_t batch, hipStream_t stream) {
    GradArgs a = {};
    a.dy = static_cast<const f16*>(dy);
    for (int l = 0; l < n; ++l) {
        a.z[l] = z ? static_cast<const f16*>(z[l]) : nullptr;
        a.scales[l] = scales ? static_cast<const f16*>(scales[l]) : nullptr;
    }
    a.dz = static_cast<f16*>(dz);
    a.levels = dz ? grad_levels(dz, n, op, batch) : nullptr;
    a.partial = partial;
    a.out = (int)out;
    a.op = (int)op;
    a.T = (int)batch;
    const int64_t chunks = grad_chunks(out, batch), n_cols = grad_level_cols(op);
    if (chunks * n_cols > INT32_MAX) return hipErrorInvalidValue;
    a.n_cols = (int)n_cols;
    const dim3 grid((unsigned)(chunks * n_cols));
    auto kern = grad_kernel(n, act, grad_wave_tokens(out, batch));
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_bias_sum(const BiasSum& b, hipStream_t stream) {
    const int64_t blocks = bias_sum_blocks(b);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(act_bias_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, b);
    return hipGetLastError();
}

}  // namespace aqlm
