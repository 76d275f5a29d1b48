// Gradients of the pre-activations, the first step of the backward passes:
//
//   one layer    dz  = dy act'(z)               (no activation: dz = dy)
//   gated        dzg = dy zu act'(zg),  dzu = dy act(zg)
//   bias         dbias[i] = sum over tokens t of dz[t][i]
//
// computed in fp32 from the fp16 inputs.  dz is rounded to fp16 once: it is the operand of
// the fp16 matrix cores in dx = dz W.  The bias sums take the fp32 values, in a fixed
// order: each wave adds its 4 tokens, a workgroup its four waves, and act_bias_kernel the
// workgroups' sums, four runs of them in order and then the runs.
//
// Elementwise, bound by HBM: 2 bytes read per input and element, 2 written.  A thread
// takes 8 consecutive rows of W, 16 bytes of each operand.
#include "act_launch.h"
#include "act_math.h"
#include "aqlm_device.h"

namespace aqlm {

namespace {

constexpr int kGradWaveTokens = 4;                   // tokens per wave, all loaded before any is used
constexpr int kGradChunk = 4 * kGradWaveTokens;      // tokens per workgroup
constexpr int kGradCols = 512;                       // columns per workgroup: 64 lanes of 8

struct GradArgs {
    const f16* dy;
    const f16* z[2];
    const f16* mant[2];
    f16* dz;
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

template <int N, int ACT>
__global__ __launch_bounds__(256) void act_grad_kernel(GradArgs a) {
    __shared__ float red[3][N][kGradCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int cb = (int)(blockIdx.x % a.n_cols), chunk = (int)(blockIdx.x / a.n_cols);
    const int c0 = cb * kGradCols + 8 * lane;
    const int t0 = chunk * kGradChunk, t1 = min(a.T, t0 + kGradChunk);
    const bool vec = a.out % 8 == 0;   // rows of 16-byte chunks
    const int left = a.out - c0;       // columns of this lane inside the matrix
    constexpr int kOps = N == 1 ? 2 : 3;   // dy, then z (gated: zg, zu)
    const int tw = t0 + wave * kGradWaveTokens, n_tok = min(kGradWaveTokens, t1 - tw);   // may be <= 0
    const bool in_row = left > 0;
    // every load of the wave's tokens first; a token past the batch repeats the last one
    f16x8 v[kGradWaveTokens][kOps];
    if (in_row && n_tok > 0) {
#pragma unroll
        for (int i = 0; i < kGradWaveTokens; ++i) {
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
            int e;
            m[l][q] = (a.mant[l] != nullptr && q < left) ? scale_mantissa((float)a.mant[l][c0 + q], &e) : 1.f;
            sum[l][q] = 0.f;
        }
    if (c0 < a.op) {
#pragma unroll
        for (int i = 0; i < kGradWaveTokens; ++i) {
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
                f16x8 o;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float w = q < left ? g[l][q] : 0.f;
                    sum[l][q] += w;
                    o[q] = (f16)(q < left ? w * m[l][q] : 0.f);
                }
                if (a.dz != nullptr)
                    *reinterpret_cast<u32x4*>(a.dz + (size_t)(tw + i) * (N * a.op) + (size_t)l * a.op + c0) = as_u32x4(o);
            }
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

// 64 sums a workgroup; wave w adds the w-th of four runs of the chunks, eight loads in flight.
__global__ __launch_bounds__(256) void act_bias_kernel(const float* __restrict__ partial, f16* d0, f16* d1, int n,
                                                       int out, int chunks) {
    __shared__ float red[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t i = (int64_t)blockIdx.x * 64 + lane, per = (int64_t)n * out;
    const int run = (chunks + 3) / 4, c1 = min(chunks, (wave + 1) * run);
    float s = 0.f;
    for (int c = wave * run; c < c1; c += 8) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = i < per && c + q < c1 ? partial[(size_t)(c + q) * per + i] : 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += v[q];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || i >= per) return;
    s = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
    if (i < out) d0[i] = (f16)s;
    else d1[i - out] = (f16)s;
}

__global__ __launch_bounds__(256) void zero16_kernel(f16* p, int64_t n) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) p[i] = (f16)0.f;
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

int64_t grad_chunks(int64_t batch) { return (batch + kGradChunk - 1) / kGradChunk; }

hipError_t launch_act_grad(const void* dy, const void* const* z, const void* const* mant, int n, int act, void* dz,
                           float* partial, void* const* dbias, int64_t out, int64_t op, int64_t batch,
                           hipStream_t stream) {
    GradArgs a = {};
    a.dy = static_cast<const f16*>(dy);
    for (int l = 0; l < n; ++l) {
        a.z[l] = z ? static_cast<const f16*>(z[l]) : nullptr;
        a.mant[l] = mant ? static_cast<const f16*>(mant[l]) : nullptr;
    }
    a.dz = static_cast<f16*>(dz);
    a.partial = partial;
    a.out = (int)out;
    a.op = (int)op;
    a.T = (int)batch;
    const int64_t chunks = grad_chunks(batch), n_cols = (op + kGradCols - 1) / kGradCols;
    if (chunks * n_cols > INT32_MAX) return hipErrorInvalidValue;
    a.n_cols = (int)n_cols;
    const dim3 grid((unsigned)(chunks * n_cols));
    void (*kern)(GradArgs) = nullptr;
    switch (act) {
        case kActRelu: kern = n == 1 ? act_grad_kernel<1, kActRelu> : act_grad_kernel<2, kActRelu>; break;
        case kActSilu: kern = n == 1 ? act_grad_kernel<1, kActSilu> : act_grad_kernel<2, kActSilu>; break;
        case kActGelu: kern = n == 1 ? act_grad_kernel<1, kActGelu> : act_grad_kernel<2, kActGelu>; break;
        case kActGeluTanh: kern = n == 1 ? act_grad_kernel<1, kActGeluTanh> : act_grad_kernel<2, kActGeluTanh>; break;
        default: kern = n == 1 ? act_grad_kernel<1, kActNone> : act_grad_kernel<2, kActNone>; break;
    }
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, stream, a);
    if (partial != nullptr) {
        const int64_t per = (int64_t)n * out;
        hipLaunchKernelGGL(act_bias_kernel, dim3((unsigned)((per + 63) / 64)), dim3(256), 0, stream, partial,
                           static_cast<f16*>(dbias[0]), n > 1 ? static_cast<f16*>(dbias[1]) : nullptr, n, (int)out,
                           (int)chunks);
    }
    return hipGetLastError();
}

}  // namespace aqlm
