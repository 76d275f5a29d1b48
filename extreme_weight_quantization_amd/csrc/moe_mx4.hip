// A mixture-of-experts layer for few tokens, experts in MX4: as moe.hip, with the products of mx4_body.h.
//
// A tile of 16 matrix-core rows is 8 rows of gate and the same 8 of up (lanes with l % 16 < 8: gate), so that one
// workgroup has both halves of h = act(zg) zu, which goes to the down product as two fp16 numbers (hidden_pair.h): there a column is two, added
// in the registers.
//
// Bound by the codes, and for small calls by what comes before the first of them (ids, the deal of items).  32 experts
// of 2048 x 1056, 40 tokens of 4: 49 us in a graph, gate and up 27 (2.7 TB/s), down 20 (1.8 TB/s), combining 3; 8 experts of 4096 x 14336,
// 1 token of 2: 54 us (3.5 TB/s).
#include <algorithm>

#include "act_math.h"
#include "moe_plan.h"
#include "mx4_body.h"
#include "mx4_launch.h"

namespace aqlm {

namespace {

constexpr int kCols = 16, kHalf = kMxRows / 2;
constexpr int kTiles = 4;   // of a group
constexpr int kMoeNk = 2;   // steps a wave holds: three spill registers where a column is two numbers, and gain nothing else

struct MoeMxProduct {
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    const f16* x;            // gate and up: [tokens][in]; down: the hidden pairs
    f16* h;                  // gate and up: [pairs][2][rows]
    float* part;             // down: [pairs][rows], before the weights
    const int32_t* ids;
    MxSteps st;
    int experts, pairs, k, rows, act;
    float fixed;
};

template <bool GATED, int NK, bool WIDE>
__global__ __launch_bounds__(kMxThreads) void moe_mx4_kernel(MoeMxProduct p) {
    __shared__ MoeLds m;
    __shared__ float red[kTiles * kMxWaves * 256];
    constexpr int kTileRows = GATED ? kHalf : kMxRows;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const MoeItems items = moe_items<kCols>(p.ids, p.pairs, p.experts, kCols, m);
    const int n = items.n;
    const int tiles = (p.rows + kTileRows - 1) / kTileRows;
    const int parts = moe_parts(n, (int)gridDim.x, tiles, p.fixed);
    for (int u = xcd_run((int)blockIdx.x, (int)gridDim.x); u < n * parts; u += (int)gridDim.x) {
        int e;
        const int cols = moe_item<false>(items, u / parts, p.pairs, p.k, kCols, m, e);
        const size_t row0 = (size_t)p.rows * e * p.st.nb;   // the expert's first block
        const int r16 = lane & 15, layer = GATED && r16 >= kHalf;
        const uint8_t* wq = (layer ? p.codes[1] : p.codes[0]) + row0 * kMxBlockBytes;
        const uint8_t* ws = (layer ? p.scales[1] : p.scales[0]) + row0;
        const int col = min(r16, cols - 1), part = u % parts;
        // One column tile, or (down, more than 8 columns) a tile of each of a pair's numbers.
        const auto product = [&](auto ct_const, auto n_const) {
            constexpr int kCt = decltype(ct_const)::value;
            constexpr bool kTogether = !GATED && kCt == 1;   // columns 2 c and 2 c + 1 are a pair's numbers
            int xrow[kCt];
            if constexpr (GATED) {
                xrow[0] = m.x[col];
            } else if constexpr (kTogether) {
                xrow[0] = 2 * m.y[min(r16 / 2, cols - 1)] + (r16 & 1);
            } else {
                xrow[0] = 2 * m.y[col];
                xrow[1] = 2 * m.y[col] + 1;
            }
            const auto fin = [&](int t0, int nt, auto sum) {
                for (int idx = tid; idx < nt * cols * kTileRows; idx += kMxThreads) {
                    const int r = idx % kTileRows, ic = idx / kTileRows, i = ic / cols, c = ic - i * cols;
                    const int row = (t0 + i * parts) * kTileRows + r;
                    if (row >= p.rows) continue;
                    if constexpr (GATED) {
                        float v[1] = {sum(i, c, r)};
                        act_values(p.act, v);
                        store_pair(v[0] * sum(i, c, r + kHalf), p.h, m.y[c], row, p.rows);
                    } else {
                        const float v = kTogether ? sum(i, 2 * c, r) + sum(i, 2 * c + 1, r) * (1.f / kPairFine) : sum(i, c, r);
                        p.part[(size_t)m.y[c] * p.rows + row] = v * kPairUnit;
                    }
                }
            };
            mx4_body<kCt, NK, kFmt16, decltype(n_const)::value, WIDE, kTileRows, kCt == 2>(
                wq, ws, mx4_rows16(p.x, p.st.nb), xrow, p.st, part, parts, tiles, red, MxTileRows{r16 & (kTileRows - 1), p.rows}, fin);
        };
        // no more tiles in a group than there are
        const auto grouped = [&](auto ct_const) {
            using std::integral_constant;
            if (tiles <= part + parts) product(ct_const, integral_constant<int, 1>{});
            else if (tiles <= part + 2 * parts) product(ct_const, integral_constant<int, 2>{});
            else product(ct_const, integral_constant<int, kTiles>{});
        };
        if constexpr (GATED) {
            grouped(std::integral_constant<int, 1>{});
        } else {
            if (cols <= kCols / 2) grouped(std::integral_constant<int, 1>{});
            else grouped(std::integral_constant<int, 2>{});
        }
    }
}

template <bool GATED>
hipError_t launch_product(MoeMxProduct p, int64_t in, hipStream_t stream) {
    int nk;
    p.st = mx4_steps(in, kMoeNk, &nk);
    auto kern = p.st.nb < kMxWideBlocks ? moe_mx4_kernel<GATED, 1, false>
                : nk == 1               ? moe_mx4_kernel<GATED, 1, true>
                                        : moe_mx4_kernel<GATED, kMoeNk, true>;
    hipLaunchKernelGGL(kern, dim3(device_cu_count()), dim3(kMxThreads), 0, stream, p);
    return hipGetLastError();
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// As moe.hip's, with 17/32 of a byte a weight and 1 us.
float start_cost(int layers, int64_t rows, int64_t in) {
    return 1.f / ((float)layers * (float)rows * (float)in * 0.53f / 20e3f);
}

}  // namespace

int64_t moe_mx4_workspace(int64_t in, int64_t inner, int64_t tokens, int64_t k) {
    return round256(tokens * k * 2 * inner * 2) + round256(tokens * k * in * 4);
}

hipError_t launch_moe_mx4(const MoeMx4Layers& L, const MoeCall& c, void* workspace, hipStream_t stream) {
    MoeMxProduct p = {};
    p.h = static_cast<f16*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + round256((int64_t)c.pairs() * 2 * c.inner * 2));
    p.x = static_cast<const f16*>(c.x);
    for (int l = 0; l < 2; ++l) {
        p.codes[l] = static_cast<const uint8_t*>(L.codes[l]);
        p.scales[l] = static_cast<const uint8_t*>(L.scales[l]);
    }
    p.ids = c.ids;
    p.experts = c.experts;
    p.pairs = c.pairs();
    p.k = c.k;
    p.rows = (int)c.inner;
    p.act = c.act;
    p.fixed = start_cost(2, c.inner, c.in);
    hipError_t r = launch_product<true>(p, c.in, stream);
    if (r != hipSuccess) return r;
    p.codes[0] = static_cast<const uint8_t*>(L.codes[2]);
    p.scales[0] = static_cast<const uint8_t*>(L.scales[2]);
    p.x = p.h;
    p.rows = (int)c.in;
    p.fixed = start_cost(1, c.inner, c.in);
    r = launch_product<false>(p, c.inner, stream);
    if (r != hipSuccess) return r;
    return launch_moe_combine(p.part, c, stream);
}

}  // namespace aqlm
