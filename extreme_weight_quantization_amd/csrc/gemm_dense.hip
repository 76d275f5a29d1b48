// Prefill product on decoded weights:  Y[t][i] = sum_k X[t][k] W16[i][k].
//
// "The AQLM Quantization Algorithm, Explained", Figure 2 of the MCQ section:
// at inference the product with the activations runs on dequantized
// half-precision weights, each the sum of the selected codewords times the
// row scale.  The two-pass prefill path first writes those weights once
// (decode_kernel, bit-exact fp16, the scale already applied) and then runs
// this dense fp16 matrix-core product over them.  Against the fused kernels,
// which decode every W tile again for each 256-token tile, it trades 2 bytes
// per weight of HBM traffic (written once, read once per XCD) for decoding
// each weight once.
//
// A workgroup owns a 256-token x 128-row output tile and walks k in steps of
// 64 inputs, each split into two k-halves of 32 for the products.  Twelve
// waves play two roles:
//   8 consumer waves  each own a 64x64 piece: they read 16-byte fragments from
//                     LDS and run 16x16x32 fp16 matrix-core products with fp32
//                     accumulators, and issue no global load;
//   4 loader waves    copy the X and W tiles of each step straight from global
//                     memory into LDS (direct-to-LDS loads), 12 loads a wave.
// With the copies in the consumer waves instead (6 loads each) the product took
// 10-13 % longer; with two loader waves, 6-9 % longer.
//
// Pipeline (one barrier per step; B_k is the barrier that ends step k):
//   step k : loaders load the X and W tiles of step k+2 (whole rows of 128
//            bytes); consumers read half 0 of step k while multiplying half 1
//            of step k-1, then read half 1 of step k while multiplying half 0;
//            B_k: the loaders' loads issued before step k have landed and the
//            consumers' fragment reads are done.
// X and W keep three whole-step stages each: 96 + 48 = 144 KB of LDS.  The
// products run in the same order as a plain k loop, so the skew changes no
// result.
//
// LDS layout of a stage: row r holds the 8 chunks (16 bytes each) of its 64
// inputs; chunk c sits in slot 8r + (c ^ ((r >> 1) & 7)).  A direct-to-LDS
// load writes 64 consecutive slots, 8 whole rows, so each load reads 8 full
// 128-byte lines (loading the two halves of a row at different times, 16 rows
// of 64 bytes per load, was measured 15-25 % slower).  The 16 lanes of a
// fragment read (16 consecutive rows, one chunk) hit 16 distinct 16-byte bank
// groups.
//
// Epilogue (out % 8 == 0): after a last barrier each consumer wave passes its 64x64 tile
// through LDS and stores whole 128-byte rows of y, 16 bytes per lane.
//
// Tile order: consecutive workgroups go to different XCDs, so workgroup b
// takes tile (b % 8) * per + b / 8 of the token-fastest tile order.  Each XCD
// then holds a contiguous run of row tiles with all their token tiles: its L2
// keeps its own W tiles, and the X tiles that its concurrent workgroups share.
//
// The same kernel with an epilogue (MODE kDenseAct, kDenseGated; see act_launch.h):
//   one layer    z = s (x w^T) + bias, y = act(z) + residual;
//   gated        the 128 rows of a tile are 64 outputs of two layers, 16 rows of the gate
//                and 16 of the up projection in turn, so one wave holds both products of
//                an output: y = act(zg) zu.
// MODE kDensePart / kDenseGatedPart: the k steps of a tile are split over `splits` workgroups,
// where the tiles alone leave CUs idle; each writes its fp32 part of the product, and
// skinny_finish_kernel (skinny.hip) adds the parts in order and runs the epilogue.  Work items
// are ordered split by split, so the items of an XCD share one range of k of x and W.
// BM: tokens of a tile, 256 next to 128 rows, or 128 next to 256 rows for batches that would
// leave half of the first kind empty.
// A wave passes its fp32 tile through LDS (64 rows of 64 + 4 floats: the writes of the four
// lane quarters, 4 rows apart, then hit distinct banks) and finishes 8 outputs a lane,
// with 16-byte accesses to y, z and the residual; everything up to the one rounding
// of y (and of z where it is kept) is fp32.
#include <algorithm>

#include "act_bias.h"
#include "act_launch.h"
#include "act_math.h"
#include "aqlm_device.h"
#include "aqlm_launch.h"

namespace aqlm {

namespace {

constexpr int kDenseBM = 256;                // tokens per tile (BM = 256; or 128 x 256)
constexpr int kDenseBN = 128;                // output rows per tile
constexpr int kDenseWaves = 8;                // consumer waves: the products
constexpr int kDenseLoaders = 4;              // loader waves: the global-to-LDS copies
constexpr int kDenseThreads = 64 * (kDenseWaves + kDenseLoaders);
constexpr int kDenseStages = 3;
constexpr size_t kDenseLds = (size_t)kDenseStages * (kDenseBM + kDenseBN) * 8 * 16;
static_assert(kDenseLds <= 163840, "LDS budget");
constexpr int kXcds = 8;                     // tile order only; any count gives correct results

// loads a loader wave issues per step: 8 of X (64 rows), 4 of W (32 rows)
constexpr int kDenseLoadsPerStep = 12;

__device__ __forceinline__ int stage_slot(int r, int c) { return 8 * r + (c ^ ((r >> 1) & 7)); }

// B_{k-1}: every load issued before the previous step has landed (the previous
// step's own stay in flight), every LDS read of the workgroup is done.
__device__ __forceinline__ void step_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kDenseLoadsPerStep));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

enum DenseMode : int { kDensePlain = 0, kDenseAct = 1, kDenseGated = 2, kDensePart = 3, kDenseGatedPart = 4 };
constexpr bool dense_gated(int mode) { return mode == kDenseGated || mode == kDenseGatedPart; }
constexpr bool dense_part(int mode) { return mode == kDensePart || mode == kDenseGatedPart; }

// What the modes with an epilogue take next to the product's arguments.
struct DenseEpi {
    const f16* w1;          // gated: the up projection's weights (w: the gate's)
    const f16* scales[2];   // row factors applied to the product, or NULL
    const f16* bias[2];
    const f16* residual;
    f16* z[2];
    int act;
    const float* units;     // one layer: factors of the tokens' products, or NULL
    float* partial;         // parts: [split][token][layer][op]
    int splits, op;
};
constexpr int kEpiRow = 68;   // floats per row of a wave's fp32 tile in LDS
static_assert((size_t)kDenseWaves * 64 * kEpiRow * sizeof(float) <= kDenseLds, "epilogue tiles");

// 8 consecutive fp16 values at p, of which `left` are inside the matrix.
__device__ __forceinline__ void epi_load8(const f16* p, int left, bool vec, float (&v)[8]) {
    if (vec) {
        const f16x8 c = *reinterpret_cast<const f16x8*>(p);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = (float)c[q];
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < left ? (float)p[q] : 0.f;
    }
}

__device__ __forceinline__ void epi_store8(f16* p, int left, bool vec, const float (&v)[8]) {
    f16x8 c;
#pragma unroll
    for (int q = 0; q < 8; ++q) c[q] = (f16)v[q];
    if (vec) {
        *reinterpret_cast<u32x4*>(p) = as_u32x4(c);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < left) p[q] = c[q];
    }
}

// The epilogue of one wave: acc[i][j] holds D[4 (l / 16) + r][l % 16] of the 16x16 block (i, j)
// of its 64x64 piece.  tok0: its first token; col0: its first output.
template <int MODE>
__device__ __forceinline__ void dense_epilogue(const f32x4 (&acc)[4][4], float* tile, int lane, int tok0, int col0,
                                               f16* y, int out, int T, const DenseEpi& e, int split) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                tile[(i * 16 + 4 * (lane >> 4) + r) * kEpiRow + j * 16 + (lane & 15)] = acc[i][j][r];
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    const bool vec = out % 8 == 0;
    // one layer: 8 lanes of 8 outputs a row; gated: 4 lanes of 8 outputs a row, the gate's in
    // columns 32 (c / 2) + 8 (c % 2) .. of the tile, the up projection's 16 further
    constexpr bool kGated = dense_gated(MODE);
    constexpr int kLanes = kGated ? 4 : 8;
    const int c = lane % kLanes;
    const int at = kGated ? 32 * (c >> 1) + 8 * (c & 1) : 8 * c;
    const int col = col0 + 8 * c, left = out - col;
    if (left <= 0) return;
    constexpr int kN = kGated ? 2 : 1;
    if constexpr (dense_part(MODE)) {   // rows of op % 8 == 0 floats: whole chunks
#pragma unroll
        for (int it = 0; it < kLanes; ++it) {
            const int rr = it * (64 / kLanes) + lane / kLanes, tok = tok0 + rr;
            if (tok >= T) continue;
#pragma unroll
            for (int l = 0; l < kN; ++l) {
                const f32x4* src = reinterpret_cast<const f32x4*>(tile + rr * kEpiRow + at + 16 * l);
                f32x4* dst = reinterpret_cast<f32x4*>(e.partial + (((size_t)split * T + tok) * kN + l) * e.op + col);
                dst[0] = src[0];
                dst[1] = src[1];
            }
        }
        return;
    }
    float s[kN][8], b[kN][8];
#pragma unroll
    for (int l = 0; l < kN; ++l)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int k = min(col + q, out - 1);
            s[l][q] = e.scales[l] != nullptr ? (float)e.scales[l][k] : 1.f;
            b[l][q] = e.bias[l] != nullptr ? (float)e.bias[l][k] : 0.f;
        }
#pragma unroll 1
    for (int it = 0; it < kLanes; ++it) {
        const int rr = it * (64 / kLanes) + lane / kLanes, tok = tok0 + rr;
        if (tok >= T) continue;
        const size_t o = (size_t)tok * out + col;
        float v[8];
        const float unit = MODE == kDenseAct && e.units != nullptr ? e.units[tok] : 1.f;
#pragma unroll
        for (int l = 0; l < kN; ++l) {
            const float* src = tile + rr * kEpiRow + at + 16 * l;
            float z[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) z[q] = src[q] * unit * s[l][q] + b[l][q];
            if (e.z[l] != nullptr) epi_store8(e.z[l] + o, left, vec, z);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = l == 0 ? z[q] : v[q] * z[q];
            if (l == 0) act_values(e.act, v);
        }
        if constexpr (MODE == kDenseAct) {
            if (e.residual != nullptr) {
                float res[8];
                epi_load8(e.residual + o, left, vec, res);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] += res[q];
            }
        }
        epi_store8(y + o, left, vec, v);
    }
}

// y carries no __restrict__: the residual may be y itself, each element read by the lane
// that then writes it.
template <int MODE, int BM>
__global__ __launch_bounds__(kDenseThreads) void gemm_dense_kernel(const f16* __restrict__ x,
                                                                   const f16* __restrict__ w, f16* y,
                                                                   int out, int in, int T, int n_tt, int n_tiles,
                                                                   int per_xcd, DenseEpi epi) {
    constexpr int BN = kDenseBM + kDenseBN - BM;                 // W rows of a tile
    constexpr int kCols = dense_gated(MODE) ? BN / 2 : BN;       // outputs per tile
    constexpr int kXStage = BM * 8, kWStage = BN * 8;            // 16-byte slots of a stage (a whole 64-input step)
    constexpr int kWOff = kDenseStages * kXStage;
    extern __shared__ u32x4 smem[];
    u32x4* Xs = smem;            // [stage 3][kXStage]
    u32x4* Ws = smem + kWOff;    // [stage 3][kWStage]
    const int item = (int)(blockIdx.x % kXcds) * per_xcd + (int)(blockIdx.x / kXcds);
    const int splits = dense_part(MODE) ? epi.splits : 1;
    if (item >= n_tiles * splits) return;   // the whole workgroup: the grid is rounded up to kXcds * per_xcd
    const int split = dense_part(MODE) ? item / n_tiles : 0, tile = dense_part(MODE) ? item % n_tiles : item;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int lw = wave - kDenseWaves;   // loader index (loader waves only)
    const int n0 = (tile / n_tt) * kCols;
    const int t0 = (tile % n_tt) * BM;
    const int n_all = in / 64;        // the launcher guarantees in % 64 == 0
    const int k_at = dense_part(MODE) ? (int)((int64_t)split * n_all / splits) : 0;   // first step of this part
    const int n_k = dense_part(MODE) ? (int)((int64_t)(split + 1) * n_all / splits) - k_at : n_all;

    // The tiles of step j into stage j % 3.  Load q writes slots 64 q .. 64 q + 63:
    // lane l fills slot 64 q + l, which holds chunk (l % 8) ^ ((r >> 1) & 7) of row
    // r = 8 q + l / 8, so the 8 lanes of a row read its whole 128-byte line.
    const int rsub = lane >> 3;
    auto load_step = [&](int j) {
        const int jc = k_at + min(j, n_k - 1);
        u32x4* dx = Xs + (j % kDenseStages) * kXStage;
        u32x4* dw = Ws + (j % kDenseStages) * kWStage;
#pragma unroll
        for (int i = 0; i < BM / 32; ++i) {
            const int q = (BM / 32) * lw + i;
            const int r = 8 * q + rsub;
            const int c = (lane & 7) ^ ((r >> 1) & 7);
            const int tok = min(t0 + r, T - 1);
            __builtin_amdgcn_global_load_lds((const void*)(x + (size_t)tok * in + (size_t)(8 * jc + c) * kGroup),
                                             lds_ptr(dx + 64 * q), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < BN / 32; ++i) {
            const int q = (BN / 32) * lw + i;
            const int r = 8 * q + rsub;
            const int c = (lane & 7) ^ ((r >> 1) & 7);
            const f16* wl = w;
            int row = min(n0 + r, out - 1);
            if constexpr (dense_gated(MODE)) {   // rows 32 m .. + 15: the gate's outputs 16 m ..; + 16: the up's
                wl = ((r >> 4) & 1) ? epi.w1 : w;
                row = min(n0 + 16 * (r >> 5) + (r & 15), out - 1);
            }
            __builtin_amdgcn_global_load_lds((const void*)(wl + (size_t)row * in + (size_t)(8 * jc + c) * kGroup),
                                             lds_ptr(dw + 64 * q), 16, 0, 0);
        }
    };

    constexpr int kWN = BN / 64;      // consumer waves across the rows
    const int wm = wave / kWN, wn = wave % kWN;
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // fragments of half h of step j: lane l holds A[l%16][8(l/16)..] and B[8(l/16)..][l%16]
    auto read_frags = [&](int j, int h, f16x8 (&a)[4], f16x8 (&b)[4]) {
        const u32x4* xb = Xs + (j % kDenseStages) * kXStage;
        const u32x4* wb = Ws + (j % kDenseStages) * kWStage;
        const int cc = 4 * h + (lane >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = as_f16x8(xb[stage_slot(wm * 64 + i * 16 + (lane & 15), cc)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = as_f16x8(wb[stage_slot(wn * 64 + i * 16 + (lane & 15), cc)]);
    };
    // 16 products of one k-half, one fragment read slotted between every two of them
    // (product, read, product: 1-7 % faster than read, product, product)
    auto mma16 = [&](const f16x8 (&a)[4], const f16x8 (&b)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = mfma16x16x32(a[i], b[j], acc[i][j]);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one matrix product
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one matrix product
        }
    };
    if (lw >= 0) {
        // loader: the same barriers as the consumers, the loads of step k+2 after B_{k-1}
        // (stage (k-1) % 3: step k-1 was read before B_{k-1})
        load_step(0);
        load_step(1);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));   // steps 0 and 1 landed
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        load_step(2);
        for (int k = 1; k < n_k; ++k) {
            step_barrier();
            load_step(k + 2);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));   // no load in flight into the epilogue's LDS
        if (MODE != kDensePlain || out % 8 == 0) {
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
        return;
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    f16x8 a0[4], b0[4], a1[4], b1[4];
    // step 0: both halves of stage 0 read, half 0 multiplied
    __builtin_amdgcn_sched_barrier(0);
    read_frags(0, 0, a0, b0);
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    read_frags(0, 1, a1, b1);
    mma16(a0, b0);
    for (int k = 1; k < n_k; ++k) {
        step_barrier();
        __builtin_amdgcn_sched_barrier(0);
        read_frags(k, 0, a0, b0);
        mma16(a1, b1);          // half 1 of step k-1
        __builtin_amdgcn_sched_barrier(0);
        read_frags(k, 1, a1, b1);
        mma16(a0, b0);          // half 0 of step k
    }
    mma16(a1, b1);              // half 1 of the last step

    if constexpr (MODE != kDensePlain) {
        // every load has landed and every fragment read is done: the stages are free
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        dense_epilogue<MODE>(acc, reinterpret_cast<float*>(smem) + wave * 64 * kEpiRow, lane, t0 + wm * 64,
                             n0 + wn * (kCols / kWN), y, out, T, epi, split);
        return;
    }
    if (out % 8 == 0) {
        // Every load of every wave has landed and every fragment read is done, so the
        // stages are free: each wave's 64x64 tile goes through LDS (fp16, rows of 64 + 8
        // padding) and leaves as 16-byte stores, 8 lanes per 128-byte row of y.
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        constexpr int kEpiStride = 72;
        f16* etile = reinterpret_cast<f16*>(smem) + wave * 64 * kEpiStride;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    etile[(i * 16 + 4 * (lane >> 4) + r) * kEpiStride + j * 16 + (lane & 15)] = (f16)acc[i][j][r];
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        const int c8 = (lane & 7) * 8;
        const int col = n0 + wn * 64 + c8;
        if (col < out) {   // out % 8 == 0: a chunk is wholly inside or wholly outside
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int rr = it * 8 + (lane >> 3);
                const int tok = t0 + wm * 64 + rr;
                if (tok < T)
                    *reinterpret_cast<u32x4*>(y + (size_t)tok * out + col) =
                        *reinterpret_cast<const u32x4*>(etile + rr * kEpiStride + c8);
            }
        }
        return;
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));   // no LDS load in flight at exit

    // rows not a multiple of 8: lane holds D[4*(l/16)+r][l%16] of block (i, j), stored directly
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = n0 + wn * 64 + j * 16 + (lane & 15);
        if (col >= out) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tok = t0 + wm * 64 + i * 16 + 4 * (lane >> 4) + r;
                if (tok < T) y[(size_t)tok * out + col] = (f16)acc[i][j][r];
            }
    }
}

// Tiles of BM tokens, dealt to the XCDs in contiguous runs.
template <int MODE, int BM>
hipError_t launch_dense(const void* x, const void* w16, void* y, int64_t out, int64_t in, int64_t batch,
                        const DenseEpi& epi, hipStream_t stream) {
    if (in % 64 != 0) return hipErrorInvalidValue;
    if (out == 0 || batch == 0) return hipSuccess;
    const hipError_t e = hipFuncSetAttribute((const void*)gemm_dense_kernel<MODE, BM>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)kDenseLds);
    if (e != hipSuccess) return e;
    constexpr int BN = kDenseBM + kDenseBN - BM, kCols = dense_gated(MODE) ? BN / 2 : BN;
    const int64_t n_tt = (batch + BM - 1) / BM;
    const int64_t n_tiles = ((out + kCols - 1) / kCols) * n_tt;
    const int64_t per = (n_tiles * (dense_part(MODE) ? epi.splits : 1) + kXcds - 1) / kXcds;
    if (per * kXcds > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_dense_kernel<MODE, BM>), dim3((unsigned)(per * kXcds)), dim3(kDenseThreads), kDenseLds,
                       stream, (const f16*)x, (const f16*)w16, (f16*)y, (int)out, (int)in, (int)batch, (int)n_tt,
                       (int)n_tiles, (int)per, epi);
    return hipGetLastError();
}

// How the product of n layers is tiled: tokens of a tile, and the workgroups that share a
// tile's k steps.  A whole launch of tiles runs in rounds of kDenseCus workgroups, each as
// long as its k steps; the split that takes the fewest microseconds by this count is
// taken, with kStepUs for a step, kRoundUs to fill and drain a round's pipeline, kFinishUs for the finishing
// launch and kPartBytesUs to write and add the parts (a plain launch has none, and stores y itself).
// Measured on 256 CUs, kernel times by the profiler: 32768 rows at 256 tokens, one round of 128 x 256 tiles, take 28,
// 47, 77 and 161 us for 16, 32, 64 and 128 steps (0.9 to 1.3 a step), 4096 rows at 200 tokens with split steps 21.6 and
// 28.2 for 64 and 128 (0.8 to 0.9 a step, start and end 3 to 9), their finishing launch 4.8 and 5.8.
struct DensePlan {
    int bm, splits;
};
constexpr int kDenseCus = 256;
constexpr double kStepUs = 0.85, kRoundUs = 3.0, kFinishUs = 3.0, kPartBytesUs = 2.5e6;

// Bytes of one part of the product of n layers.
int64_t part_bytes(int n, int64_t out, int64_t batch) { return batch * n * ((out + 7) / 8 * 8) * 4; }

DensePlan dense_plan(int n, int64_t out, int64_t in, int64_t batch) {
    DensePlan best = {kDenseBM, 1};
    double best_us = 1e300;
    const int64_t n_k = in / 64, part = part_bytes(n, out, batch);
    for (int bm = 128; bm <= 256; bm += 128) {
        if (bm == 128 && batch > 1024) continue;
        const int64_t cols = (kDenseBM + kDenseBN - bm) / n;
        const int64_t tiles = (out + cols - 1) / cols * ((batch + bm - 1) / bm);
        for (int s = 1; s <= kMaxSplits && s <= n_k; ++s) {
            if (s > 1 && s * part > kPartsRoom) break;
            const int64_t rounds = (tiles * s + kDenseCus - 1) / kDenseCus, steps = (n_k + s - 1) / s;
            double us = (double)rounds * ((double)steps * kStepUs + kRoundUs);
            if (s > 1) us += kFinishUs + (double)s * batch * n * out * 8 / kPartBytesUs;
            if (us < best_us) {
                best_us = us;
                best = {bm, s};
            }
        }
    }
    return best;
}

}  // namespace

hipError_t launch_gemm_dense(const void* x, const void* w16, void* y, int64_t out, int64_t in, int64_t batch,
                             hipStream_t stream) {
    return launch_dense<kDensePlain, kDenseBM>(x, w16, y, out, in, batch, DenseEpi{}, stream);
}

int64_t dense_partial_bytes(int n, int64_t out, int64_t kp, int64_t batch) {
    const int64_t splits = std::min<int64_t>(kMaxSplits, kp / 64);
    return splits < 2 ? 0 : std::min(splits * part_bytes(n, out, batch), kPartsRoom);
}

hipError_t launch_gemm_dense_act(const void* x, const void* const* w, const void* const* scales, int n,
                                 const Epilogue& epi, void* partial, int64_t out, int64_t kp, int64_t batch,
                                 const BiasSum& bias, hipStream_t stream) {
    const DensePlan p = dense_plan(n, out, kp, batch);
    DenseEpi e = {};
    for (int l = 0; l < n; ++l) {
        e.scales[l] = scales ? static_cast<const f16*>(scales[l]) : nullptr;
        e.bias[l] = static_cast<const f16*>(epi.bias[l]);
        e.z[l] = static_cast<f16*>(epi.z[l]);
    }
    e.residual = static_cast<const f16*>(epi.residual);
    e.act = epi.act;
    e.units = epi.units;
    e.w1 = n == 2 ? static_cast<const f16*>(w[1]) : nullptr;
    e.partial = static_cast<float*>(partial);
    e.splits = p.splits;
    e.op = (int)((out + 7) / 8 * 8);
    if (p.splits == 1) {
        const hipError_t b = launch_bias_sum(bias, stream);
        if (b != hipSuccess) return b;
        if (n == 2)
            return p.bm == 128 ? launch_dense<kDenseGated, 128>(x, w[0], epi.y, out, kp, batch, e, stream)
                               : launch_dense<kDenseGated, 256>(x, w[0], epi.y, out, kp, batch, e, stream);
        return p.bm == 128 ? launch_dense<kDenseAct, 128>(x, w[0], epi.y, out, kp, batch, e, stream)
                           : launch_dense<kDenseAct, 256>(x, w[0], epi.y, out, kp, batch, e, stream);
    }
    hipError_t r;
    if (n == 2)
        r = p.bm == 128 ? launch_dense<kDenseGatedPart, 128>(x, w[0], nullptr, out, kp, batch, e, stream)
                        : launch_dense<kDenseGatedPart, 256>(x, w[0], nullptr, out, kp, batch, e, stream);
    else
        r = p.bm == 128 ? launch_dense<kDensePart, 128>(x, w[0], nullptr, out, kp, batch, e, stream)
                        : launch_dense<kDensePart, 256>(x, w[0], nullptr, out, kp, batch, e, stream);
    if (r != hipSuccess) return r;
    return launch_finish(n, e.partial, scales, epi, out, e.op, batch, p.splits, bias, stream);
}

}  // namespace aqlm
