// Host-side launchers of the fused products (epilogue, gated) and their backward passes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "aqlm_launch.h"

namespace aqlm {

struct BiasSum;   // act_bias.h

// Workspaces never shrink as the batch grows, so that one sized for the largest batch serves all: the
// *_bytes functions below give room for any batch up to theirs, in closed form or as the largest over its steps.
// Where a product's sum is split into fp32 parts, at most kPartsRoom bytes of them are written (or one
// part, if that is more and the product always writes one): a limit that only products larger than a full chip's
// tiles feel (over a grid of layers and batches the planned times rise by 0.02 % on average, 7 % at most).
constexpr int kMaxSplits = 32;
constexpr int64_t kPartsRoom = (int64_t)128 << 20;

// Workgroups go to the 8 XCDs in turn: the place of workgroup b of n in an order in which each XCD
// has a contiguous run, so that neighbours in it share an L2 (any count gives correct results).
__device__ __forceinline__ int xcd_run(int b, int n) {
    constexpr int kX = 8;
    const int x = b % kX;
    return x * (n / kX) + (x < n % kX ? x : n % kX) + b / kX;
}

// What follows the product of one or two layers that share x.  One layer:
// z = W x + bias, y = act(z) + residual.  Two layers (gate, up): zg, zu likewise,
// y = act(zg) zu.  Absent pointers are NULL.  residual may be y itself.
struct Epilogue {
    const void* bias[2];       // fp16 [out]
    const void* residual;      // fp16 [batch][out]
    void* z[2];                // fp16 [batch][out]: where the pre-activations are kept
    void* y;                   // fp16 [batch][out]
    int act;
    const float* units = nullptr;   // [batch]: factors of the tokens' products, powers of two (NULL: ones)
};

// Gradients dz of `batch` tokens as launch_act_grad writes them (dz NULL: none).
struct GradRows {
    void* dz = nullptr;
    int64_t batch = 0;
};

// One or two layers (n) of the same scheme, out and in.
struct ActLayers {
    const void* codes[2];
    const void* codebooks[2];
    const void* scales[2];
    int n;
    GradRows grads = {};   // launch_decode_transposed: the rows that it brings to one unit beside its own work
};

// How a decoded weight enters the fp16 workspace: the codewords' fp32 sum times the row
// scale; or the sum alone (M = 1: exact; the scale then goes into the epilogue, or into dz).
enum class WeightScale : int { kFull = 0, kNone = 1 };

// w[l][row][0 .. kp) for l < n: the layers' fp16 weights, inputs past `in` zero (kp % 8 == 0).
hipError_t launch_decode_rows(const GenericScheme& sc, const ActLayers& L, WeightScale ws, void* const* w,
                              int64_t out, int64_t in, int64_t kp, hipStream_t stream);
// wt[k][l * op + row] for k < in, l < n, row < op: the transposed weights, rows past `out`
// zero (op % 64 == 0).  L.grads: every row of dz is brought to the unit of its largest level
// before the product sums over it, and the units are written to grad_units.
hipError_t launch_decode_transposed(const GenericScheme& sc, const ActLayers& L, WeightScale ws, void* wt,
                                    int64_t out, int64_t in, int64_t op, hipStream_t stream);
// xp[t][0 .. kp): x [batch][in], inputs past `in` zero.
hipError_t launch_pad_rows(const void* x, void* xp, int64_t batch, int64_t in, int64_t kp, hipStream_t stream);

// Zeros in n 16-bit elements at p (a kernel: a memset may not be recorded into a graph).
hipError_t launch_zero16(void* p, int64_t n, hipStream_t stream);

// The dense product of gemm_dense.hip on fp16 weights w[l] [out][kp] with an epilogue:
// z_l = scales[l] (x w_l^T) + bias_l (scales NULL: 1).  partial: dense_partial_bytes bytes,
// for shapes whose k steps are split over workgroups.
int64_t dense_partial_bytes(int n, int64_t out, int64_t kp, int64_t batch);
hipError_t launch_gemm_dense_act(const void* x, const void* const* w, const void* const* scales, int n,
                                 const Epilogue& epi, void* partial, int64_t out, int64_t kp, int64_t batch,
                                 const BiasSum& bias, hipStream_t stream);

// y from fp32 parts of the products, [part][token][layer][op]: the parts added in order,
// then scales (NULL: 1) and the epilogue.  bias: sums that further workgroups of the launch add.
hipError_t launch_finish(int n, const float* partial, const void* const* scales, const Epilogue& epi, int64_t out,
                         int64_t op, int64_t batch, int parts, const BiasSum& bias, hipStream_t stream);

// Gradients of the pre-activations, fp16, as the dense product's x: dz[t][l * op + i] for
// i < op (rows past `out` zero).  One layer: dy act'(z); two: dy zu act'(zg) and dy act(zg).
// scales: row scales that multiply them in fp32 (NULL: none).
// dz is in units of 2^(20 level) (act_math.h); behind it, each 256-byte aligned, lie the levels
// [batch][n][grad_level_cols(op)] of the blocks of 512 rows, and room for one unit a token.
// partial: fp32 [grad_chunks(out, batch)][n][out]: sums over chunks of tokens of the unscaled
// fp32 gradients (NULL: not wanted); launch_bias_sum, or the launch that finishes a
// product from parts, adds the chunks.
inline int64_t grad_level_cols(int64_t op) { return (op + 511) / 512; }
inline int64_t grad_align(int64_t bytes) { return (bytes + 255) / 256 * 256; }
inline int8_t* grad_levels(void* dz, int n, int64_t op, int64_t batch) {
    return static_cast<int8_t*>(dz) + grad_align(batch * n * op * 2);
}
inline float* grad_units(void* dz, int n, int64_t op, int64_t batch) {
    return reinterpret_cast<float*>(grad_levels(dz, n, op, batch) + grad_align(batch * n * grad_level_cols(op)));
}
int64_t grad_chunks(int64_t out, int64_t batch);
// Tokens per wave: 4, or 1 where that leaves fewer than two workgroups a CU (8 tokens of 4096 gated rows: 10.2 us
// with 4, 6.0 with 1).
constexpr int kGradCols = 512, kGradFew = 512;
inline int grad_wave_tokens(int64_t out, int64_t batch) {
    return (out + kGradCols - 1) / kGradCols * ((batch + 15) / 16) < kGradFew ? 1 : 4;
}
// The most chunks of any batch up to this one: of it, or of the last with one token a wave.
inline int64_t grad_chunks_room(int64_t out, int64_t batch) {
    if (out < 1) return 0;
    const int64_t one = (kGradFew - 1) / ((out + kGradCols - 1) / kGradCols) * 16;
    const int64_t few = ((batch < one ? batch : one) + 3) / 4, many = (batch + 15) / 16;
    return few > many ? few : many;
}
hipError_t launch_act_grad(const void* dy, const void* const* z, const void* const* scales, int n, int act, void* dz,
                           float* partial, int64_t out, int64_t op, int64_t batch, hipStream_t stream);
hipError_t launch_bias_sum(const BiasSum& b, hipStream_t stream);

// The products of batch 1..16 (gemv_act.hip): any scheme, no workspace.
hipError_t launch_gemv_act(const GenericScheme& sc, const ActLayers& L, const void* x, const Epilogue& epi, int64_t out,
                           int64_t in, int64_t batch, hipStream_t stream);
// Their streaming form (gemv_stream.hip): false where it does not serve the call (as
// gemv_stream_lds), else true with the launch's result.
struct GemvEpi;
bool launch_gemv_stream_act(const ActLayers& L, const GemvEpi& epi, const void* x, void* y, int64_t out, int64_t in,
                            int64_t batch, hipStream_t stream, hipError_t* result);

// The products of tens to hundreds of tokens (skinny.hip), 2x8, 1x16 and 4x8 g16: straight from the codes, with
// fp32 partial sums in the workspace.  The work is dealt to at most kSkinnyWorkgroups
// workgroups, a fixed number so that the sums' order does not depend on the device.
constexpr int kSkinnyWorkgroups = 256;
constexpr int kSkinnyMaxBatch2x8 = 512, kSkinnyMaxBatch2x8Gated = 384;
constexpr int kSkinnyMaxBatch1x16 = 256, kSkinnyMaxBatch1x16Few = 128;   // Few: of layers with few units
constexpr int kSkinnyMaxBatch4x8 = 320, kSkinnyMaxBatch4x8Gated = 256;
// The largest batch of n layers, by scheme (one of the three).
inline int skinny_max_batch(const GenericScheme& sc, int n) {
    if (sc.M == 1) return kSkinnyMaxBatch1x16;
    if (sc.M == 2) return n == 2 ? kSkinnyMaxBatch2x8Gated : kSkinnyMaxBatch2x8;
    return n == 2 ? kSkinnyMaxBatch4x8Gated : kSkinnyMaxBatch4x8;
}
bool skinny_serves(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch);
int64_t skinny_partial_bytes(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch);
hipError_t launch_skinny(const GenericScheme& sc, const ActLayers& L, const void* x, void* partial, const Epilogue& epi,
                         int64_t out, int64_t in, int64_t batch, hipStream_t stream);

// dx of some tens of tokens (skinny_back.hip), 2x8, 1x16 and 4x8 g16: straight from the codes, dz as
// launch_act_grad writes it with the scales, fp32 parts in the workspace.
constexpr int kSkinnyBackMaxBatch2x8 = 256;
constexpr int kSkinnyBackMaxBatch1x16 = 128;
constexpr int kSkinnyBackMaxBatch4x8 = 128;
bool skinny_back_serves(const GenericScheme& sc, int64_t out, int64_t in, int64_t batch);
int64_t skinny_back_partial_bytes(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch);
// skinny_back_grads: the shapes whose dz and bias sums the product computes itself, from grads
// (then not NULL; dz and bias are not used).
struct BackGrads {
    const void* dy;
    const void* z[2];
    void* dbias[2];
    int act;
};
bool skinny_back_grads(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch);
hipError_t launch_skinny_back(const GenericScheme& sc, const ActLayers& L, const void* dz, const BackGrads* grads,
                              void* partial, void* dx, int64_t out, int64_t in, int64_t op, int64_t batch,
                              const BiasSum& bias, hipStream_t stream);

// The slice-list product of one layer, or of gate and up, batch 1, with the epilogue in its
// reduction (gemv_lists.hip).  L as for launch_gemv_lists_fused; its y is not used.
hipError_t launch_lists_act(ListsLayers L, const void* x, const Epilogue& epi, int64_t in, hipStream_t stream);

}  // namespace aqlm
