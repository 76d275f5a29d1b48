// A mixture-of-experts layer for few tokens, experts in MX4: as moe.hip, with the products of mx4_body.h.
//
// A tile of 16 matrix-core rows is 8 rows of gate and the same 8 of up (lanes with l % 16 < 8: gate), so that one
// workgroup has both halves of h = act(zg) zu; four neighbouring tiles are one block of 32 hidden values, which goes
// to the down product in the four-piece form of mx4.h, from fp32: it is rounded by 2^-19 of the block's largest only.  The
// splitting takes a thread some 2000 clocks a block, so up to kHold blocks wait for it in LDS.
//
// Bound by the codes, and for small calls by what comes before the first of them (ids, the deal of items, the split of x).  32 experts
// of 2048 x 1056, 40 tokens of 4: 49 us in a graph, gate and up 27 (2.7 TB/s), down 20 (1.8 TB/s), combining 3; 8 experts of 4096 x 14336,
// 1 token of 2: 63 us (3.0 TB/s).
#include <algorithm>

#include "act_math.h"
#include "moe_plan.h"
#include "mx4_body.h"
#include "mx4_launch.h"

namespace aqlm {

namespace {

// Steps a wave holds: a fourth spills registers beside the deal of items, and scratch costs a launch about 3 us.
constexpr int kMxMoeNk = 3, kCols = 16, kHalf = kMxRows / 2;
constexpr int kDownTiles = 4;
constexpr int kHold = 4;   // blocks of hidden values that wait to be split together, a thread a column
// Activations that are split inside the product (100 KB of LDS): a launch of its own for the split costs 5 us.
constexpr int kInlineBlocks = 1024;
bool split_inline(int64_t tokens, int64_t in) { return std::min<int64_t>(tokens, kCols) * (in / kMxBlock) <= kInlineBlocks; }

struct MoeMxProduct {
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    char* x;                 // split records of the input
    char* h;                 // gate and up: of the hidden vectors of the pairs
    float* part;             // down: [pairs][rows], before the weights
    const int32_t* ids;
    MxSteps st;
    int experts, pairs, k, rows, act;
    int cols;                // INLINE: columns that LDS has room for
    float fixed;
};

// INLINE (gate and up): p.x is fp16 rows, and each workgroup splits those of its item into LDS, at most kInlineBlocks blocks.  An item
// has no more pairs than there are tokens then; an expert that a token names twice may have more, which are an item of their own.
template <bool GATED, bool INLINE, bool WIDE>
__global__ __launch_bounds__(kMxThreads) void moe_mx4_kernel(MoeMxProduct p) {
    extern __shared__ u32x4 smem[];
    __shared__ MoeLds m;
    __shared__ float red[mx4_red_floats(1)];
    __shared__ float hb[kHold][kCols][kMxBlock + 1];
    constexpr int kNk = WIDE ? kMxMoeNk : 1;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int most = INLINE ? p.cols : kCols;   // pairs of an item
    const MoeItems items = moe_items<kCols>(p.ids, p.pairs, p.experts, most, m);
    const int n = items.n;
    const int tiles = GATED ? (p.rows + kHalf - 1) / kHalf : (p.rows + kMxRows - 1) / kMxRows;
    const int parts = moe_parts(n, (int)gridDim.x, GATED ? (tiles + 3) / 4 : tiles, p.fixed);
    for (int u = xcd_run((int)blockIdx.x, (int)gridDim.x); u < n * parts; u += (int)gridDim.x) {
        int e;
        const int cols = moe_item<false>(items, u / parts, p.pairs, p.k, most, m, e);
        const size_t row0 = (size_t)p.rows * e * p.st.nb;   // the expert's first block
        const int r16 = lane & 15, layer = GATED && r16 >= kHalf;
        const uint8_t* wq = (layer ? p.codes[1] : p.codes[0]) + row0 * kMxBlockBytes;
        const uint8_t* ws = (layer ? p.scales[1] : p.scales[0]) + row0;
        const int col = min(r16, cols - 1);
        const int xrow[1] = {INLINE ? col : GATED ? (int)m.x[col] : (int)m.y[col]};
        const int part = u % parts, nb = p.st.nb;
        const MxInputRows<kFmt6> xin = {INLINE ? SplitRows{reinterpret_cast<char*>(smem), cols, nb} : SplitRows{p.x, kSplitTokens, nb}};
        if constexpr (INLINE) {
            for (int i = tid; i < cols * nb; i += kMxThreads) {
                const int c = i / nb;
                uint32_t o[kSplitDwords], s;
                split_block(load_block16(reinterpret_cast<const f16*>(p.x) + ((size_t)m.x[c] * nb + (i - c * nb)) * kMxBlock), o, s);
                store_split(xin.rows, c, i - c * nb, o, s);
            }
            __syncthreads();
        }
        const auto prepare = []() {};
        const auto row_of = [&](int tile) { return min(GATED ? tile * kHalf + (r16 & (kHalf - 1)) : tile * kMxRows + r16, p.rows - 1); };
        if constexpr (GATED) {
            // blocks part, part + parts, ... of the hidden vectors, kHold at a time; the products' registers are free when the
            // blocks are split
            for (int b0 = part; b0 * 4 < tiles; b0 += kHold * parts) {
                const int end = min(tiles, 4 * (b0 + kHold * parts));
                mx4_body<1, kNk, kFmt6, true, 4, WIDE>(
                    wq, ws, xin, xrow, p.st, b0, parts, end, red, row_of, prepare,
                    [&](int t0, int, auto sum) {
                        const int slot = (t0 / 4 - b0) / parts;
                        for (int idx = tid; idx < cols * kMxBlock; idx += kMxThreads) {   // rows is a multiple of 32: whole blocks
                            const int c = idx / kMxBlock, i = idx % kMxBlock;
                            float v[1] = {sum(i / kHalf, c, i % kHalf)};
                            act_values(p.act, v);
                            hb[slot][c][i] = v[0] * sum(i / kHalf, c, i % kHalf + kHalf);
                        }
                    });
                const int held = ((end + 3) / 4 - b0 + parts - 1) / parts;
                if (tid < held * cols) {
                    const int q = tid / cols, c = tid - q * cols;
                    f32x16 even, odd;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        even[i] = hb[q][c][2 * i];
                        odd[i] = hb[q][c][2 * i + 1];
                    }
                    uint32_t o[kSplitDwords], s;
                    split_block32(even, odd, o, s);
                    store_split(SplitRows{p.h, kSplitTokens, p.rows / kMxBlock}, m.y[c], b0 + q * parts, o, s);
                }
                __syncthreads();
            }
        } else {
            mx4_body<1, kNk, kFmt6, false, kDownTiles, WIDE>(
                wq, ws, xin, xrow, p.st, part, parts, tiles, red, row_of, prepare,
                [&](int t0, int nt, auto sum) {
                    for (int idx = tid; idx < nt * cols * kMxRows; idx += kMxThreads) {
                        const int r = idx % kMxRows, ic = idx / kMxRows, i = ic / cols, c = ic - i * cols;
                        const int row = (t0 + i * parts) * kMxRows + r;
                        if (row < p.rows)
                            p.part[(size_t)m.y[c] * p.rows + row] = sum(i, c, r);
                    }
                });
        }
    }
}

template <bool GATED, bool INLINE, bool WIDE>
hipError_t launch_v(const MoeMxProduct& p, int lds, hipStream_t stream) {
    auto kern = moe_mx4_kernel<GATED, INLINE, WIDE>;
    if (INLINE) {
        const hipError_t r = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (r != hipSuccess) return r;
    }
    hipLaunchKernelGGL(kern, dim3(device_cu_count()), dim3(kMxThreads), lds, stream, p);
    return hipGetLastError();
}

template <bool GATED, bool INLINE>
hipError_t launch_product(const MoeMxProduct& p, int lds, hipStream_t stream) {
    return p.st.nb >= kMxWideBlocks ? launch_v<GATED, INLINE, true>(p, lds, stream) : launch_v<GATED, INLINE, false>(p, lds, stream);
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// As moe.hip's, with 17/32 of a byte a weight and 1 us.
float start_cost(int layers, int64_t rows, int64_t in) {
    return 1.f / ((float)layers * (float)rows * (float)in * 0.53f / 20e3f);
}

}  // namespace

int64_t moe_mx4_workspace(int64_t in, int64_t inner, int64_t tokens, int64_t k) {
    const int64_t pairs = tokens * k;
    return round256(mx4_split_bytes(tokens, in)) + round256(mx4_split_bytes(pairs, inner)) + round256(pairs * in * 4);
}

hipError_t launch_moe_mx4(const MoeMx4Layers& L, const MoeCall& c, void* workspace, hipStream_t stream) {
    char* at = static_cast<char*>(workspace);
    auto take = [&](int64_t bytes) {
        char* p = at;
        at += bytes;
        return p;
    };
    MoeMxProduct p = {};
    const bool inlined = split_inline(c.tokens, c.in);
    if (!inlined) p.x = take(round256(mx4_split_bytes(c.tokens, c.in)));
    p.h = take(round256(mx4_split_bytes(c.pairs(), c.inner)));
    p.part = reinterpret_cast<float*>(at);
    hipError_t r = hipSuccess;
    if (inlined) p.x = const_cast<char*>(static_cast<const char*>(c.x));
    else r = launch_mx4_split(c.x, p.x, c.in, c.tokens, stream);
    if (r != hipSuccess) return r;
    for (int l = 0; l < 2; ++l) {
        p.codes[l] = static_cast<const uint8_t*>(L.codes[l]);
        p.scales[l] = static_cast<const uint8_t*>(L.scales[l]);
    }
    p.ids = c.ids;
    p.st = mx4_steps(c.in, kMxMoeNk);
    p.experts = c.experts;
    p.pairs = c.pairs();
    p.k = c.k;
    p.rows = (int)c.inner;
    p.act = c.act;
    p.fixed = start_cost(2, c.inner, c.in);
    p.cols = std::min(c.tokens, kCols);
    const int lds = inlined ? SplitRows::record_bytes(p.cols) * (int)(c.in / kMxBlock) : 0;
    r = inlined ? launch_product<true, true>(p, lds, stream) : launch_product<true, false>(p, lds, stream);
    if (r != hipSuccess) return r;
    p.codes[0] = static_cast<const uint8_t*>(L.codes[2]);
    p.scales[0] = static_cast<const uint8_t*>(L.scales[2]);
    p.x = p.h;
    p.st = mx4_steps(c.inner, kMxMoeNk);
    p.rows = (int)c.in;
    p.fixed = start_cost(1, c.inner, c.in);
    r = launch_product<false, false>(p, 0, stream);
    if (r != hipSuccess) return r;
    return launch_moe_combine(p.part, c, stream);
}

}  // namespace aqlm
