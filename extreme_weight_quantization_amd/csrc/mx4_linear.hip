// Products of MX4 weights: y = act(W x + bias) + residual.
//
// z[t][i] = sum over blocks b of 2^(s_ib - 127) sum_k q_ibk x[t][32 b + k].  The scaled matrix instruction takes the codes
// and their scales as they lie in memory; x is in MX4 too, or in fp16 as four 6-bit pieces (mx4.h), so a weight costs no
// vector instruction.
//
// Few tokens (mx4_rows_kernel): the codes are read once, 17/32 of a byte a weight, and that bounds the time.  Matrix-core
// rows are output rows, columns are tokens; a workgroup keeps the activations of all inputs in the registers of its 8 waves
// (100 bytes a block and token: 12 KB of a wave's 64 KB for each step of 128 inputs and 16 tokens) and streams the rows
// past them (mx4_body.h); with one or two tiles a workgroup it reads them from LDS.  1 token: 8192 -> 28672 29 us (4.3 TB/s),
// 4096 -> 4096 5.7 in a graph (1.6 TB/s: latencies); 16 tokens 8192 -> 28672 38 us.
#include <algorithm>

#include "act_math.h"
#include "mx4_body.h"
#include "mx4_gemm.h"
#include "mx4_launch.h"

namespace aqlm {

namespace {

struct MxEpilogue {
    const f16* bias;
    const f16* residual;   // may be y
    f16* y;
    int act;
};

// Activations that are split inside the product: at most this many blocks of 32, 1.2 KB of LDS for every 12.  A launch
// of its own for the split costs more from there down.
// Blocks of x that a workgroup splits itself, into 100 KB of LDS; a launch of its own for the split costs 3 us (4096 -> 4096: 8 tokens
// 8.5 us without, 16 tokens 9.1 with it).
constexpr int kInlineBlocks = 1024;

template <int CT, int NK, int FMT, bool INLINE, bool WIDE = false, int TILES = mx4_tiles(CT)>
__global__ __launch_bounds__(kMxThreads) void mx4_rows_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, const void* x,
                                                              const void* xs, MxSteps st, int out, int T, MxEpilogue e) {
    extern __shared__ u32x4 smem[];
    float* red = reinterpret_cast<float*>(smem);
    const int lane = threadIdx.x & (kWave - 1);
    const int col0 = (int)blockIdx.y * CT * 16, cols = min(T - col0, CT * 16);
    int xrow[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) xrow[t] = min(col0 + t * 16 + (lane & 15), T - 1);
    const int n_tiles = (out + kMxRows - 1) / kMxRows;
    MxInputRows<FMT> xin;
    if constexpr (FMT == kFmt4) {
        xin = {static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(xs), st.nb};
    } else if constexpr (INLINE) {
        xin.rows = SplitRows{reinterpret_cast<char*>(red + mx4_red_floats(CT)), T, st.nb};
    } else {
        xin.rows = SplitRows{static_cast<char*>(const_cast<void*>(x)), kSplitTokens, st.nb};
    }
    // Blocks that this thread splits, asked for in front of the first codes: loads come back in order.
    constexpr int kMine = INLINE ? kInlineBlocks / kMxThreads : 1;
    f16x32 mine[kMine];
    if constexpr (INLINE) {
#pragma unroll
        for (int q = 0; q < kMine; ++q)
            mine[q] = load_block16(static_cast<const f16*>(x) + (size_t)min((int)threadIdx.x + q * kMxThreads, T * st.nb - 1) * kMxBlock);
    }
    const int nwg = (int)gridDim.x;
    const auto row_of = [&](int tile) { return min(tile * kMxRows + (lane & 15), out - 1); };
    const auto prepare = [&]() {
        if constexpr (INLINE) {
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int i = threadIdx.x + q * kMxThreads;
                if (i >= T * st.nb) break;
                uint32_t o[kSplitDwords], s;
                split_block(mine[q], o, s);
                store_split(xin.rows, i / st.nb, i % st.nb, o, s);
            }
            __syncthreads();
        }
    };
    const auto fin = [&](int t0, int n, auto sum) {
        for (int idx = threadIdx.x; idx < n * cols * kMxRows; idx += kMxThreads) {
            const int r = idx % kMxRows, ic = idx / kMxRows, i = ic / cols, col = ic - i * cols;
            const int row = (t0 + i * nwg) * kMxRows + r;
            if (row >= out) continue;
            float v[1] = {sum(i, col, r)};
            if (e.bias != nullptr) v[0] += (float)e.bias[row];
            act_values(e.act, v);
            const size_t at = (size_t)(col0 + col) * out + row;
            if (e.residual != nullptr) v[0] += (float)e.residual[at];
            e.y[at] = (f16)v[0];
        }
    };
    if constexpr (INLINE && WIDE && TILES <= 2) {
        mx4_body_lds<NK, TILES>(codes, scales, xin.rows, xrow[0], st, (int)blockIdx.x, nwg, n_tiles, red, row_of, prepare, fin);
    } else {
        mx4_body<CT, NK, FMT, false, TILES, WIDE>(codes, scales, xin, xrow, st, (int)blockIdx.x, nwg, n_tiles, red, row_of, prepare,
                                                  fin);
    }
}

struct RowsCall {
    const void *codes, *scales, *x, *xs;
    MxEpilogue e;
    int64_t out, in;
    int T;
    hipStream_t stream;
};

template <int CT, int NK, int FMT, bool INLINE, bool WIDE = false, int TILES = mx4_tiles(CT)>
hipError_t launch_rows_v(const RowsCall& c) {
    auto kern = mx4_rows_kernel<CT, NK, FMT, INLINE, WIDE, TILES>;
    const MxSteps st = mx4_steps(c.in, NK);
    const size_t lds = mx4_red_floats(CT) * sizeof(float) +
                       (INLINE ? (size_t)SplitRows::record_bytes(c.T) * st.nb : 0);
    if (lds > 65536) {
        const hipError_t r = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (r != hipSuccess) return r;
    }
    const int tiles = (int)((c.out + kMxRows - 1) / kMxRows), groups = (c.T + CT * 16 - 1) / (CT * 16);
    hipLaunchKernelGGL(kern, dim3(std::min(tiles, device_cu_count()), groups), dim3(kMxThreads), lds, c.stream,
                       static_cast<const uint8_t*>(c.codes), static_cast<const uint8_t*>(c.scales), c.x, c.xs, st,
                       (int)c.out, c.T, c.e);
    return hipGetLastError();
}

// x split in LDS: one or two tiles a workgroup by mx4_body_lds, more by mx4_body, which keeps x in registers (4096 -> 4096 at 1 token
// 5.7 us against 6.4, 4096 -> 8192 6.4 against 7.3; four tiles and more: 4096 -> 28672 17.6 against 16.3).
template <int NK>
hipError_t launch_inline(const RowsCall& c) {
    return (c.out + kMxRows - 1) / kMxRows <= device_cu_count() ? launch_rows_v<1, NK, kFmt6, true, true, 1>(c)
                                                                : launch_rows_v<1, NK, kFmt6, true, true, 2>(c);
}

template <int FMT, bool INLINE>
hipError_t launch_rows(const RowsCall& c) {
    if constexpr (!INLINE) {
        if (c.T > 32) return launch_rows_v<4, 1, FMT, INLINE>(c);
        if (c.T > 16) return launch_rows_v<2, 2, FMT, INLINE>(c);
    }
    if (c.in < kMxWideBlocks * kMxBlock) return launch_rows_v<1, 1, FMT, INLINE>(c);
    if constexpr (INLINE) {
        if ((c.out + kMxRows - 1) / kMxRows <= 2 * device_cu_count()) {
            switch (mx4_steps(c.in, 4).nk) {
                case 1: return launch_inline<1>(c);
                case 2: return launch_inline<2>(c);
                case 3: return launch_inline<3>(c);
                default: return launch_inline<4>(c);
            }
        }
    }
    return launch_rows_v<1, 4, FMT, INLINE, true>(c);
}

bool split_inline(int64_t in, int64_t batch) { return batch <= 16 && batch * (in / kMxBlock) <= kInlineBlocks; }

}  // namespace

int64_t mx4_linear_workspace(bool x_mx4, int64_t out, int64_t in, int64_t batch) {
    if (out == 0 || batch == 0) return 0;
    const int64_t split = x_mx4 || split_inline(in, batch) ? 0 : mx4_split_bytes(batch, in);
    return split + (mx4_gemm_serves(x_mx4, out, in, batch) ? mx4_gemm_part_bytes(out, in, batch) : 0);
}

hipError_t launch_mx4_linear(const void* codes, const void* scales, MxInput x, const Epilogue& e, void* workspace,
                             int64_t out, int64_t in, int64_t batch, hipStream_t stream) {
    const bool four = x.scales != nullptr, inlined = !four && split_inline(in, batch);
    char* part = static_cast<char*>(workspace);
    if (!four && !inlined) {
        const hipError_t r = launch_mx4_split(x.x, workspace, in, batch, stream);
        if (r != hipSuccess) return r;
        x.x = workspace;
        part += mx4_split_bytes(batch, in);
    }
    if (mx4_gemm_serves(four, out, in, batch)) return launch_mx4_gemm(codes, scales, x, e, part, out, in, batch, stream);
    const RowsCall c = {codes, scales, x.x, x.scales,
                        MxEpilogue{static_cast<const f16*>(e.bias[0]), static_cast<const f16*>(e.residual),
                                   static_cast<f16*>(e.y), e.act},
                        out, in, (int)batch, stream};
    if (four) return launch_rows<kFmt4, false>(c);
    return inlined ? launch_rows<kFmt6, true>(c) : launch_rows<kFmt6, false>(c);
}

}  // namespace aqlm
