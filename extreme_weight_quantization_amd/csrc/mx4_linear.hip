// Products of MX4 weights: y = act(W x + bias) + residual.
//
// z[t][i] = sum over blocks b of 2^(s_ib - 127) sum_k q_ibk x[t][32 b + k].  With x in MX4 the scaled matrix instruction takes
// codes and scales of both as they lie in memory; with x in fp16 the codes are converted to fp16, which is exact (mx4.h).
//
// Few tokens (mx4_rows_kernel): the codes are read once, 17/32 of a byte a weight, and that bounds the time.  Matrix-core
// rows are output rows, columns are tokens; a workgroup keeps the activations of all inputs in LDS or in the registers of its 8
// waves and streams the rows past them (mx4_body.h).  1 token: 8192 -> 28672 27.6 us in a graph (4.5 TB/s), 4096 -> 4096 5.2 (1.7 TB/s:
// latencies); 16 tokens 8192 -> 28672 34 us.
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

// How fp16 activations come: STAGED, up to 16 rows in LDS, where they fit; else, to 16 rows, in records of them, made by
// mx4_records_kernel in a launch before, which 16 lanes read next to each other where rows would be 16 lines; else as they lie in memory.
// us, 16 tokens, as they lie | so: 4096 -> 28672 in LDS 27 | 19.5, 8192 -> 11008 in records 21.6 | 17.7.
template <int CT, int NK, int FMT, bool WIDE, int TILES, bool STAGED>
__global__ __launch_bounds__(kMxThreads) void mx4_rows_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, MxInputRows<FMT> xin,
                                                              MxSteps st, int out, int T, MxEpilogue e) {
    extern __shared__ u32x4 smem[];
    __shared__ float red[TILES * kMxWaves * CT * 256];
    static_assert(sizeof(red) + (STAGED ? MxStaged::kSteps * 256 : 0) <= 163840, "the LDS of a CU");
    const int lane = threadIdx.x & (kWave - 1);
    const int col0 = (int)blockIdx.y * CT * 16, cols = min(T - col0, CT * 16);
    int xrow[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) xrow[t] = min(col0 + t * 16 + (lane & 15), T - 1);
    const int n_tiles = (out + kMxRows - 1) / kMxRows;
    const int nwg = (int)gridDim.x;
    const MxStaged staged = {smem, lds_address(smem), MxStaged::row_steps(st.nb)};
    if constexpr (STAGED) staged.send(xin.x, T, st.nb);
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
    mx4_body<CT, NK, FMT, TILES, WIDE, kMxRows, false, STAGED>(codes, scales, xin, xrow, st, (int)blockIdx.x, nwg, n_tiles, red,
                                                               MxTileRows{lane & 15, out}, fin, staged);
}

// Up to 16 rows of x to records: piece e of 8 values of block b of row r at (4 b + e) * 16 + r; rows past the last repeat it.
__global__ __launch_bounds__(256) void mx4_records_kernel(const f16* __restrict__ x, u32x4* __restrict__ to, int T, int in) {
    const int i = (int)blockIdx.x * 256 + (int)threadIdx.x;   // 16 consecutive pieces of a row are read by 16 lanes each
    const int piece = i % 16 + i / 256 * 16, r = i / 16 % 16;
    if (piece < in / 8) to[(size_t)piece * 16 + r] = load16(x + (size_t)min(r, T - 1) * in + piece * 8);
}
constexpr int kRecordRows = 16;

struct RowsCall {
    const void *codes, *scales, *x, *xs;
    MxEpilogue e;
    int64_t out, in;
    int T;
    hipStream_t stream;
    bool records;   // x is in records
};

template <int CT, int NK, int FMT, bool WIDE, int TILES, bool STAGED>
hipError_t launch_rows_v(const RowsCall& c, const MxSteps& st) {
    auto kern = mx4_rows_kernel<CT, NK, FMT, WIDE, TILES, STAGED>;
    MxInputRows<FMT> x;
    if constexpr (FMT == kFmt4) x = {static_cast<const uint8_t*>(c.x), static_cast<const uint8_t*>(c.xs), st.nb};
    else if (c.records) x = {static_cast<const f16*>(c.x), 8, kRecordRows * kMxBlock, kRecordRows * 8};
    else x = mx4_rows16(static_cast<const f16*>(c.x), st.nb);
    const size_t lds = STAGED ? (size_t)c.T * MxStaged::row_steps(st.nb) * 256 : 0;
    if (lds > 0) {
        const hipError_t r = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (r != hipSuccess) return r;
    }
    const int tiles = (int)((c.out + kMxRows - 1) / kMxRows), groups = (c.T + CT * 16 - 1) / (CT * 16);
    hipLaunchKernelGGL(kern, dim3(std::min(tiles, device_cu_count()), groups), dim3(kMxThreads), lds, c.stream,
                       static_cast<const uint8_t*>(c.codes), static_cast<const uint8_t*>(c.scales), x, st, (int)c.out, c.T, c.e);
    return hipGetLastError();
}

// Steps a wave holds: four, where registers allow.
template <int CT, int FMT, bool WIDE, int TILES, bool STAGED>
hipError_t launch_rows_t(const RowsCall& c) {
    constexpr int kNk = CT == 4 ? 1 : CT == 2 ? 2 : !WIDE ? 1 : FMT == kFmt16 && TILES > (STAGED ? 3 : 2) ? 2 : 4;
    int nk;
    const MxSteps st = mx4_steps(c.in, kNk, &nk);
    if constexpr (kNk == 4) {
        if (nk == 4) return launch_rows_v<CT, 4, FMT, WIDE, TILES, STAGED>(c, st);
    }
    if constexpr (kNk >= 3) {
        if (nk == 3) return launch_rows_v<CT, 3, FMT, WIDE, TILES, STAGED>(c, st);
    }
    if constexpr (kNk >= 2) {
        if (nk == 2) return launch_rows_v<CT, 2, FMT, WIDE, TILES, STAGED>(c, st);
    }
    return launch_rows_v<CT, 1, FMT, WIDE, TILES, STAGED>(c, st);
}

// No more tiles in a group than a workgroup has: fewer leave registers for more steps in flight (4096 -> 11008, 3 tiles a workgroup, 1 and
// 16 tokens: groups of 3 tiles and 4 steps 8.3 and 10.6 us, of 4 and 2 8.9 and 11.4; 8192 -> 22016, 6 tiles, 1 token: 22.3 and 25.2).  More
// groups than of 4 tiles cost more than that (8192 -> 28672, 7 tiles, 1 token: 30.6 and 27.6).
template <int CT, int FMT, bool WIDE, bool STAGED = false>
hipError_t launch_rows_ct(const RowsCall& c) {
    const int tiles = (int)((c.out + kMxRows - 1) / kMxRows), cus = device_cu_count();
    if (tiles <= cus) return launch_rows_t<CT, FMT, WIDE, 1, STAGED>(c);
    if (tiles <= 2 * cus || mx4_tiles(CT) == 2) return launch_rows_t<CT, FMT, WIDE, 2, STAGED>(c);
    if constexpr (STAGED) {
        const int n = (tiles + cus - 1) / cus;   // of a workgroup
        if ((n + 2) / 3 == (n + 3) / 4) return launch_rows_t<CT, FMT, WIDE, 3, STAGED>(c);
    }
    return launch_rows_t<CT, FMT, WIDE, mx4_tiles(CT), STAGED>(c);
}

bool wide(int64_t in) { return in >= kMxWideBlocks * kMxBlock; }
bool fits_lds(int64_t in, int64_t batch) { return batch * ((in + 127) / 128) <= MxStaged::kSteps; }
bool in_records(int64_t in, int64_t batch) { return wide(in) && batch <= 16 && !fits_lds(in, batch); }

template <int FMT>
hipError_t launch_rows(const RowsCall& c) {
    if (c.T > 32) return launch_rows_ct<4, FMT, false>(c);
    if (c.T > 16) return launch_rows_ct<2, FMT, false>(c);
    if (!wide(c.in)) return launch_rows_ct<1, FMT, false>(c);
    if constexpr (FMT == kFmt16) {
        // few short rows are read as they lie: no wait for LDS in front of few tiles (512 -> 8192, 1 token: 3.9 us, staged 4.9)
        const bool few = c.T <= 4 && c.in <= 4096 && c.out <= (int64_t)2 * kMxRows * device_cu_count();
        if (!c.records && !few) return launch_rows_ct<1, FMT, true, true>(c);
    }
    return launch_rows_ct<1, FMT, true>(c);
}

// Room for records: what any batch up to this one may need.
int64_t records_bytes(bool x_mx4, int64_t in, int64_t batch) {
    return !x_mx4 && wide(in) && !fits_lds(in, std::min<int64_t>(batch, 16)) ? kRecordRows * in * 2 : 0;
}

}  // namespace

int64_t mx4_linear_workspace(bool x_mx4, int64_t out, int64_t in, int64_t batch) {
    if (out == 0 || batch == 0) return 0;
    const int64_t parts = mx4_gemm_serves(x_mx4, out, in, batch) ? mx4_gemm_part_bytes(out, in, batch) : 0;
    return std::max(parts, records_bytes(x_mx4, in, batch));
}

hipError_t launch_mx4_linear(const void* codes, const void* scales, MxInput x, const Epilogue& e, void* workspace,
                             int64_t out, int64_t in, int64_t batch, hipStream_t stream) {
    const bool four = x.scales != nullptr;
    if (mx4_gemm_serves(four, out, in, batch)) return launch_mx4_gemm(codes, scales, x, e, workspace, out, in, batch, stream);
    RowsCall c = {codes, scales, x.x, x.scales,
                  MxEpilogue{static_cast<const f16*>(e.bias[0]), static_cast<const f16*>(e.residual),
                             static_cast<f16*>(e.y), e.act},
                  out, in, (int)batch, stream, !four && in_records(in, batch)};
    if (c.records) {
        hipLaunchKernelGGL(mx4_records_kernel, dim3((unsigned)((in / 8 + 15) / 16)), dim3(256), 0, stream, static_cast<const f16*>(x.x),
                           static_cast<u32x4*>(workspace), (int)batch, (int)in);
        const hipError_t r = hipGetLastError();
        if (r != hipSuccess) return r;
        c.x = workspace;
    }
    return four ? launch_rows<kFmt4>(c) : launch_rows<kFmt16>(c);
}

}  // namespace aqlm
