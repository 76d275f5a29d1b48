// Gradients of a small batch with respect to the inputs, straight from the codes, 2x8, 1x16 and
// 4x8 g16:
//   dx[t][k] = sum over layers and rows i of dz[t][i] s[i] Wc[i][k].
//
// "The AQLM Quantization Algorithm, Explained", Figure 2 of the MCQ section (a group's weights
// are the sum of one codeword per codebook, times the row's scale).  The sum runs over the
// rows of W, while a codeword holds 8 inputs of one row, and the matrix cores want 8
// consecutive summed indices in a lane.  So a lane looks up the codewords of 8 consecutive
// rows at one group and transposes the 8 x 8 block in registers (v_perm_b32 pairs two rows'
// halves: 32 for 64 weights): operand t then holds input t of the group for the 8 rows.  A wave
// covers 16 groups x 32 rows with 8 operands, each multiplied by the dz of up to 64 tokens (1x16:
// 128), and no weight is ever written to memory.
//
//  * The row scale is in dz (act_grad.hip), which is rounded to fp16 anyway, and the codewords are
//    multiplied as they are, one by one for 2x8 and 4x8 g16, so no weight is rounded.
//  * dz of a token comes in units of 2^(20 level), one level per 512 rows (act_math.h).  The sums of
//    a token are kept at its highest level in the workgroup's rows (a lane has one token per column tile),
//    blocks at a lower one are brought to it as they are used, and the sums leave in units of one.
//  * A workgroup of 8 waves (4 at 128 tokens) owns 16 groups (128 inputs) of dx and a part of the rows of one
//    layer; its waves take the chunks of 32 rows in turn, each with the next chunk's codes and dz
//    in flight and no barrier, and add their sums in LDS in wave order.  Its fp32 part of dx goes to
//    the workspace; skinny_finish_kernel adds the parts in order and rounds once.
//  * GRAD: where that is little work (skinny_back_grads) the kernel takes dy and the
//    pre-activations themselves.  A lane computes the 8 gradients of its operand from 16 bytes of
//    each, every workgroup anew, and the workgroups of the first 16 groups add them over the
//    tokens for the bias.  That saves a launch and dz's way through memory.  Levels are then found chunk by
//    chunk, and a higher one brings the sums to its unit.
//  * 2x8 codebooks: LDS, 8 replicas, read without bank conflicts as in gemv.hip; 4x8 g16: 2
//    replicas of the four, no conflicts either, since neighbouring groups read different
//    halves.  1x16 codewords are gathered from L2, a chunk ahead.
//  * Neighbouring 16-group columns share lines of codes (128 bytes hold 64 groups), so they run
//    on one XCD (xcd_run): 4096x11008 1x16 at 20 tokens 38.3 -> 36.5 us.
//
// What bounds it.  1x16: the gathers (4096x11008 at 77 tokens, main kernel 44 us by the
// profiler: 5.6 M gathers, 21 us at the 264 G/s of a kernel of nothing else; without gathers it
// took 18 us less, without reloading dz 6; three chunks of codes and dz in flight
// changed nothing).  2x8: transposes, products and latencies; gated 4096x11008 at 64 tokens
// 34.3 us.
//
// Against decoding the transposed weights first (decode_work.hip), us in a graph: 4x8 g16 4096^2
// at 16 tokens 14.2 and 29.5, 4096x11008 at 128 64.7 and 72.3, at 256 108 and 80: to 128 tokens.
// 2x8 4096x11008 at 256 60 and 78, at 512 101 and 93, gated at 256 108 and 146, at 320 158 and 156: to 256.  1x16 at 128
// 54 and 79, at 192 85 and 83: to 128.
#include <algorithm>
#include <type_traits>

#include "act_bias.h"
#include "act_launch.h"
#include "act_math.h"
#include "aqlm_device.h"

namespace aqlm {

namespace {

// Waves of a workgroup by its column tiles of tokens: 8, or 4 with twice the registers a lane, which
// hold the sums of 128 tokens (1x16: one gather of a code serves them all).
constexpr int back_waves(int ct) { return ct == 8 ? 4 : 8; }
constexpr int kBGroups = 16;                                 // groups a workgroup
constexpr int kBRows = 32;                                   // rows a chunk
constexpr int kBCbBytes = 2 * kCodewords2x8 * 8 * 16;         // 64 KB: 8 replicas

// Inputs t of the groups whose sums share the LDS at a time (128 KB at most).
constexpr int back_half(int ct) { return ct >= 4 ? 4 : 8; }

struct BackArgs {
    const uint8_t* codes[2];
    const f16* codebooks[2];
    const f16* scales[2];
    const f16* dz;      // [t][l * op + i], times the scales; zero for i >= out
    const int8_t* levels;   // [t][l][level_cols]
    int level_cols;
    float* partial;     // [part][t][ip]
    int out, op, G, T, n, ip, n_cb, splits;
    // GRAD: dz is computed here
    const f16* dy;
    const f16* z[2];
    f16* dbias[2];      // NULL: not wanted
    int act;
};

__device__ __forceinline__ u32x4 lds16(uint32_t byte) {
    return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((uintptr_t)byte);
}

__device__ const u32x4 back_zero = {0u, 0u, 0u, 0u};

template <int SCHEME, int CT, bool GRAD>
__global__ __launch_bounds__(64 * back_waves(CT))
    __attribute__((amdgpu_waves_per_eu(back_waves(CT) / 4, back_waves(CT) / 4))) void skinny_back_kernel(const BackArgs a) {
    constexpr int kBWaves = back_waves(CT), kBThreads = 64 * kBWaves;
    extern __shared__ u32x4 smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lrow = lane & 15, kq = lane >> 4;
    const int item = xcd_run((int)blockIdx.x, (int)gridDim.x);
    const int cb = item % a.n_cb, rest = item / a.n_cb;
    const int split = rest % a.splits, l = (rest / a.splits) % a.n, tt = rest / (a.splits * a.n);
    constexpr bool kCbLds = SCHEME != kScheme1x16, kFour = SCHEME == kSchemeB8M4;
    constexpr int kCodewords = kFour ? 4 : 2;   // of a weight, from LDS
    // the codes of a group of 8 inputs are 2 bytes, those of a 4x8 g16 group (two of them) 4
    using Code = std::conditional_t<kFour, uint32_t, uint16_t>;
    const Code* codes = reinterpret_cast<const Code*>(l ? a.codes[1] : a.codes[0]);
    const f16* codebooks = l ? a.codebooks[1] : a.codebooks[0];
    const f16* scales = l ? a.scales[1] : a.scales[0];
    const int n_chunks = a.op / kBRows;
    const int c_end = (int)((int64_t)(split + 1) * n_chunks / a.splits);
    const int c0 = (int)((int64_t)split * n_chunks / a.splits) + wave;
    const int j = min(cb * kBGroups + lrow, a.G - 1);   // groups past the row repeat the last (not used)
    const size_t ldz = (size_t)a.n * a.op;
    const f16* dzl = a.dz + (size_t)l * a.op;

    // What a chunk needs from memory: the codes and scales of the lane's 8 rows, dz of its
    // tokens.  One set of registers: each part of the next chunk is loaded after its last use in this one.
    Code code[8];
    f16 scale[8];   // GRAD
    u32x4 dz[CT];
    int level[CT], top[CT];   // of the tokens: of dz, and of their sums
#pragma unroll
    for (int i = 0; i < CT; ++i) level[i] = top[i] = kLevelMin;
    auto row0 = [&](int c) { return min(c, n_chunks - 1) * kBRows + 8 * kq; };
    auto load_codes = [&](int c) {   // rows past the layer repeat its last one (masked when used)
#pragma unroll
        for (int r = 0; r < 8; ++r) code[r] = codes[((size_t)min(row0(c) + r, a.out - 1) * a.G + j) / (kFour ? 2 : 1)];
    };
    auto load_scales = [&](int c) {
#pragma unroll
        for (int r = 0; r < 8; ++r) scale[r] = scales[min(row0(c) + r, a.out - 1)];
    };
    auto level_at = [&](int i) -> size_t {   // tokens past the batch repeat the last (their sums are not used)
        return ((size_t)min((tt * CT + i) * 16 + lrow, a.T - 1) * a.n + l) * a.level_cols;
    };
    u32x4 raw[3] = {};   // GRAD: dy, and the pre-activations, of the lane's rows (out % 8 == 0: all inside or all past)
    auto load_dz = [&](int c) {   // tokens past the batch repeat the last (their sums are not used)
        if constexpr (GRAD) {
            const size_t at = (size_t)min(lrow, a.T - 1) * a.out + min(row0(c), a.out - 8);
            raw[0] = load16(a.dy + at);
            if (a.n == 2 || a.act != kActNone) raw[1] = load16(a.z[0] + at);
            if (a.n == 2 && l == 0) raw[2] = load16(a.z[1] + at);
        } else {
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                dz[i] = load16(dzl + (size_t)min((tt * CT + i) * 16 + lrow, a.T - 1) * ldz + row0(c));
                level[i] = a.levels[level_at(i) + min(c, n_chunks - 1) / (kLevelCols / kBRows)];
            }
        }
    };
    f32x4 acc[8][CT];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < CT; ++i) acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    // The highest level of each token in the rows of this part; the quarters take the blocks in turn.
    auto load_tops = [&]() {
        if constexpr (!GRAD) {
            const int b1 = (c_end - 1) / (kLevelCols / kBRows);
            for (int b = (int)((int64_t)split * n_chunks / a.splits) / (kLevelCols / kBRows) + kq; b <= b1; b += 4)
#pragma unroll
                for (int i = 0; i < CT; ++i) top[i] = max(top[i], (int)a.levels[level_at(i) + b]);
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                top[i] = max(top[i], __shfl_xor(top[i], 16, 64));
                top[i] = max(top[i], __shfl_xor(top[i], 32, 64));
            }
        }
    };
    // Brings dz to the level of the sums.
    auto settle_dz = [&]() {
        if constexpr (!GRAD) {
            bool differ = false;
#pragma unroll
            for (int i = 0; i < CT; ++i) differ |= level[i] != top[i];
            if (__any(differ)) {
#pragma unroll
                for (int i = 0; i < CT; ++i) dz[i] = raise_level(dz[i], top[i] - level[i]);
            }
        }
    };
    // GRAD: dz from raw, fp32 until its one rounding, at the sums' level; the bias sums of a chunk's rows
    auto make_dz = [&](int c) {
        const f16x8 dy = as_f16x8(raw[0]), z0 = as_f16x8(raw[1]), z1 = as_f16x8(raw[2]);
        float g[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) g[r] = (float)z0[r];
        if (l == 0) act_slopes(a.act, g);   // none: ones
        else act_values(a.act, g);
        const bool inside = row0(c) < a.out && lrow < a.T;
        float scaled[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            g[r] *= (float)dy[r];
            if (a.n == 2 && l == 0) g[r] *= (float)z1[r];
            g[r] = inside ? g[r] : 0.f;
            scaled[r] = inside ? g[r] * (float)scale[r] : 0.f;
        }
        // the four quarters hold the token's other rows
        float largest = largest_finite(scaled);
        largest = fmaxf(largest, __shfl_xor(largest, 16, 64));
        largest = fmaxf(largest, __shfl_xor(largest, 32, 64));
        const int now = max(top[0], grad_level(largest));
        if (__any(now != top[0])) {   // the sums to the unit of a higher level
            const float unit = level_unit(top[0] - now);
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[t][0][q] *= unit;
        }
        top[0] = now;
        const float unit = level_unit(-now);
        f16x8 o;
#pragma unroll
        for (int r = 0; r < 8; ++r) o[r] = (f16)(scaled[r] * unit);
        dz[0] = as_u32x4(o);
        if (cb == 0 && a.dbias[0] != nullptr) {   // the 16 lanes of a quarter hold the tokens of its 8 rows
            f16* db = (l ? a.dbias[1] : a.dbias[0]) + row0(c);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float s = g[r];
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
                if (lrow == 0 && row0(c) < a.out) db[r] = (f16)s;
            }
        }
    };
    const uint32_t mA = (lane >> 3) & 1u, r16 = (lane & 7u) * 16u;
    const uint32_t base = (r16 + 128u * mA) | ((r16 + 128u * (mA ^ 1u)) << 8);
    // 4x8 g16: 16 lanes (halves h of a codeword, codebooks in rotation, replicas r) hit all 16 bank groups; byte
    // i: the slot of the lane's i-th codebook in a codeword's 256 bytes
    const uint32_t rot = (lane >> 1) & 3u, rep = 128u * (lane & 1u) + 16u * ((lane >> 3) & 1u);
    const uint32_t base4 = (32u * rot + rep) | ((32u * ((rot + 1u) & 3u) + rep) << 8) |
                           ((32u * ((rot + 2u) & 3u) + rep) << 16) | ((32u * ((rot + 3u) & 3u) + rep) << 24);
    // the products of one codeword per row (w: rows 0..7 of the lane)
    auto multiply = [&](const u32x4 (&w)[8]) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            u32x4 lo, hi;   // inputs 2d and 2d + 1 of the 8 rows
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                lo[p] = __builtin_amdgcn_perm(w[2 * p + 1][d], w[2 * p][d], 0x05040100u);
                hi[p] = __builtin_amdgcn_perm(w[2 * p + 1][d], w[2 * p][d], 0x07060302u);
            }
#pragma unroll
            for (int i = 0; i < CT; ++i) acc[2 * d][i] = mfma16x16x32(as_f16x8(lo), as_f16x8(dz[i]), acc[2 * d][i]);
#pragma unroll
            for (int i = 0; i < CT; ++i)
                acc[2 * d + 1][i] = mfma16x16x32(as_f16x8(hi), as_f16x8(dz[i]), acc[2 * d + 1][i]);
        }
    };

    load_codes(c0);
    if constexpr (GRAD) load_scales(c0);
    load_dz(c0);
    if constexpr (!kCbLds) load_tops();   // next to the loads before it; LDS codebooks: to theirs
    if constexpr (kCbLds) {
        // 2x8: slot (2 k + m) 8 + r, codeword k of codebook m; 4x8 g16: slot 16 k + 8 h + 2 m + r, half h of it
#pragma unroll
        for (int it = 0; it < kBCbBytes / 16 / kBThreads; ++it) {
            const int slot = it * kBThreads + tid;
            const f16* src = kFour ? codebooks + (size_t)((slot >> 1 & 3) * kCodewords2x8 + (slot >> 4)) * 16 + (slot >> 3 & 1) * 8
                                   : codebooks + (size_t)((slot >> 3 & 1) * kCodewords2x8 + (slot >> 4)) * kGroup;
            __builtin_amdgcn_global_load_lds((const void*)src, lds_ptr(smem + it * kBThreads + wave * kWave), 16, 0, 0);
        }
        load_tops();
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
        __syncthreads();
        for (int c = c0; c < c_end; c += kBWaves) {
            u32x4 w[8];
            if constexpr (GRAD) make_dz(c);
            settle_dz();
#pragma unroll
            for (int m = 0; m < kCodewords; ++m) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if constexpr (kFour) {
                        const uint32_t d = __builtin_amdgcn_alignbit(code[r], code[r], 8u * rot);
                        w[r] = lds16(__builtin_amdgcn_perm(base4, d, 0x0c0c0004u + 0x0101u * m));
                        continue;
                    }
                    const uint32_t sel = m == 0 ? 0x0c0c0004u | (mA << 8) : 0x0c0c0005u | ((mA ^ 1u) << 8);
                    w[r] = lds16(__builtin_amdgcn_perm(base, (uint32_t)code[r], sel));
                }
                if ((c + 1) * kBRows > a.out) {   // rows past the layer count as zero
#pragma unroll
                    for (int r = 0; r < 8; ++r) w[r] = row0(c) + r < a.out ? w[r] : u32x4{0u, 0u, 0u, 0u};
                }
                if (m == kCodewords - 1) {
                    load_codes(c + kBWaves);
                    if constexpr (GRAD) load_scales(c + kBWaves);
                }
                multiply(w);
                __builtin_amdgcn_sched_barrier(0);
            }
            load_dz(c + kBWaves);
        }
    }
    if constexpr (SCHEME == kScheme1x16) {
        // the gathers of the next chunk are in flight while this one is multiplied
        u32x4 next[8];
        auto gather = [&](int c) {   // rows past the layer: zeros
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const f16* src = codebooks + (size_t)code[r] * kGroup;
                next[r] = load16(row0(c) + r < a.out ? src : reinterpret_cast<const f16*>(&back_zero));
            }
        };
        if (c0 < c_end) {
            gather(c0);
            load_codes(c0 + kBWaves);
            int c = c0;
            for (; c + kBWaves < c_end; c += kBWaves) {
                if constexpr (GRAD) make_dz(c);
                settle_dz();
                u32x4 w[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) w[r] = next[r];
                gather(c + kBWaves);
                load_codes(c + 2 * kBWaves);
                if constexpr (GRAD) load_scales(c + kBWaves);
                multiply(w);
                __builtin_amdgcn_sched_barrier(0);
                load_dz(c + kBWaves);
            }
            if constexpr (GRAD) make_dz(c);
            settle_dz();
            multiply(next);
        }
    }

    // The waves' sums, in LDS [wave][t][i][r][lane], added in wave order; kH inputs t at a time.
    // Thread (combination (i, r) of its wave, lane): group 4 kq + r, token 16 i + lane % 16.
    constexpr int kH = back_half(CT);
    // The sums' units: GRAD, of the wave, applied as it writes them; else the workgroup's, behind the sums.
    float* red = reinterpret_cast<float*>(smem);
    float* units = red + kBWaves * kH * CT * 4 * 64;
    if (!GRAD && wave == 0 && kq == 0) {
#pragma unroll
        for (int i = 0; i < CT; ++i) units[16 * i + lrow] = level_unit(top[i]);
    }
    const size_t part = (size_t)((l * a.splits) + split);
#pragma unroll
    for (int h = 0; h < 8 / kH; ++h) {
        __syncthreads();   // the codebooks, or the half before, are read
#pragma unroll
        for (int t = 0; t < kH; ++t)
#pragma unroll
            for (int i = 0; i < CT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    red[(((wave * kH + t) * CT + i) * 4 + r) * 64 + lane] =
                        GRAD ? acc[h * kH + t][i][r] * level_unit(top[i]) : acc[h * kH + t][i][r];
        __syncthreads();
        for (int q = wave; q < 4 * CT; q += kBWaves) {
            const int i = q >> 2, r = q & 3;
            const int tok = (tt * CT + i) * 16 + lrow, grp = cb * kBGroups + 4 * kq + r;
            float s[kH];
#pragma unroll
            for (int t = 0; t < kH; ++t) {
                s[t] = 0.f;
#pragma unroll
                for (int w = 0; w < kBWaves; ++w) s[t] += red[(((w * kH + t) * CT + i) * 4 + r) * 64 + lane];
                if (!GRAD) s[t] *= units[16 * i + lrow];
            }
            if (tok < a.T) {
                f32x4* dst = reinterpret_cast<f32x4*>(a.partial + (part * a.T + tok) * a.ip + 8 * (size_t)grp + h * kH);
#pragma unroll
                for (int k = 0; k < kH / 4; ++k) dst[k] = f32x4{s[4 * k], s[4 * k + 1], s[4 * k + 2], s[4 * k + 3]};
            }
        }
    }
}

struct BackPlan {
    int ct, n_tt, n_cb, splits;
};

// Token tiles of 16, 32 or 64 tokens, or 128 for 1x16.  The rows are split over as many workgroups as take the
// fewest microseconds: rounds of one workgroup a CU, each some time to start and end and
// chunk_us per chunk of a wave (1x16: 4096 gathers of the workgroup's waves, at the rate a CU gets), then the parts,
// written and added.  Measured on 256 CUs, 4096 and 8192 rows of 32768 inputs, one workgroup a CU (kernel times by the
// profiler): 2x8 at 16, 32 and 64 tokens 24.0 and 41.6, 30.1 and 51.4, 41.9 and 74.2 us, which is 1.1, 1.3 and 2.0 a
// chunk; 4x8 g16 at 16 and 64 1.8 and 4.4; 1x16 at 16, 64 and 128 4.7, 5.3 and 3.1; 4 to 10 to start and end.
// Bytes of one part of dx of n layers (their parts lie side by side).
int64_t part_bytes(int n, int64_t n_cb, int64_t batch) { return n * batch * n_cb * kBGroups * kGroup * 4; }

BackPlan back_plan(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch) {
    const bool two = sc.B == 8;   // 2x8, 4x8 g16
    BackPlan p;
    p.ct = batch <= 16 ? 1 : batch <= 32 ? 2 : batch <= 64 || two ? 4 : 8;
    p.n_tt = (int)((batch + 16 * p.ct - 1) / (16 * p.ct));
    p.n_cb = (int)((in / kGroup + kBGroups - 1) / kBGroups);
    const int64_t n_chunks = (out + 63) / 64 * 2, wgs = (int64_t)p.n_cb * n * p.n_tt, waves = back_waves(p.ct);
    const double chunk_us = two ? (p.ct == 4 ? 1.8 : 1.2) : p.ct == 8 ? 3.0 : 4.5;
    const double part_us = 0.15 * n + (double)n * batch * p.n_cb * kBGroups * kGroup * 8 / 3e6;
    double best = 1e300;
    p.splits = 1;
    const int64_t part = part_bytes(n, p.n_cb, batch);
    for (int s = 1; s <= kMaxSplits && s <= n_chunks; ++s) {
        if (s > 1 && s * part > kPartsRoom) break;
        const int64_t rounds = (wgs * s + kSkinnyWorkgroups - 1) / kSkinnyWorkgroups;
        const double us = rounds * ((double)((n_chunks + waves * s - 1) / (waves * s)) * chunk_us + 4.0) + s * part_us;
        if (us < best) {
            best = us;
            p.splits = s;
        }
    }
    return p;
}

template <int SCHEME, int CT, bool GRAD = false>
hipError_t launch_back(const BackArgs& a, int grid, hipStream_t stream) {
    auto kern = skinny_back_kernel<SCHEME, CT, GRAD>;
    constexpr size_t sums = (size_t)back_waves(CT) * back_half(CT) * CT * 4 * 64 * 4;
    constexpr size_t lds = sums + 16 * CT * 4;   // and a unit a token
    static_assert(SCHEME == kScheme1x16 || sums >= kBCbBytes, "the units lie behind the codebooks");
    static_assert(lds <= 163840, "LDS budget");
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * back_waves(CT)), lds, stream, a);
    return hipGetLastError();
}

template <int SCHEME>
hipError_t launch_ct(int ct, const BackArgs& a, int grid, hipStream_t stream) {
    if constexpr (SCHEME == kScheme1x16) {
        if (ct == 8) return launch_back<SCHEME, 8>(a, grid, stream);
    }
    if (a.dy != nullptr) return launch_back<SCHEME, 1, true>(a, grid, stream);
    return ct == 1 ? launch_back<SCHEME, 1>(a, grid, stream)
         : ct == 2 ? launch_back<SCHEME, 2>(a, grid, stream) : launch_back<SCHEME, 4>(a, grid, stream);
}

}  // namespace

bool skinny_back_serves(const GenericScheme& sc, int64_t out, int64_t in, int64_t batch) {
    const bool two = sc.M == 2 && sc.B == 8 && sc.g == 8, one = sc.M == 1 && sc.B == 16 && sc.g == 8;
    const bool four = sc.M == 4 && sc.B == 8 && sc.g == 16;
    return (two || one || four) && batch <= (two ? kSkinnyBackMaxBatch2x8 : one ? kSkinnyBackMaxBatch1x16 : kSkinnyBackMaxBatch4x8);
}

int64_t skinny_back_partial_bytes(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch) {
    const int64_t part = part_bytes(n, (in / kGroup + kBGroups - 1) / kBGroups, batch);
    return std::max(part, std::min(std::min<int64_t>(kMaxSplits, (out + 63) / 64 * 2) * part, kPartsRoom));
}

// Where a wave of a full chip has few chunks: a launch saved is 1.5 to 3.5 us, while every chunk's
// gradients, computed in each of the in / 128 groups, cost a 2x8 wave 0.5 to 1 us.  Gated, 8 tokens, us with
// and without: 2x8 4096x2048 (2 chunks a wave) 12.7 and 14.5, 4096^2 (4) silu 16.7 and 17.0, gelu 20.9 and 17.7; 1x16
// 4096^2 (4) 27.0 and 30.4, 4096x6144 (6) silu 39.5 and 41.1, gelu 43.1 and 41.5.
bool skinny_back_grads(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch) {
    const int64_t chunks = (out + kBRows - 1) / kBRows * n * ((in / kGroup + kBGroups - 1) / kBGroups);
    return batch <= 16 && out % 8 == 0 && chunks <= (sc.B == 8 ? 2 : 4) * kSkinnyWorkgroups * back_waves(1);
}

hipError_t launch_skinny_back(const GenericScheme& sc, const ActLayers& L, const void* dz, const BackGrads* grads,
                              void* partial, void* dx, int64_t out, int64_t in, int64_t op, int64_t batch,
                              const BiasSum& bias, hipStream_t stream) {
    const BackPlan p = back_plan(sc, L.n, out, in, batch);
    BackArgs a = {};
    for (int l = 0; l < L.n; ++l) {
        a.codes[l] = static_cast<const uint8_t*>(L.codes[l]);
        a.codebooks[l] = static_cast<const f16*>(L.codebooks[l]);
        a.scales[l] = static_cast<const f16*>(L.scales[l]);
    }
    a.dz = static_cast<const f16*>(dz);
    if (dz != nullptr) {
        a.levels = grad_levels(const_cast<void*>(dz), L.n, op, batch);
        a.level_cols = (int)grad_level_cols(op);
    }
    if (grads != nullptr) {
        a.dy = static_cast<const f16*>(grads->dy);
        for (int l = 0; l < L.n; ++l) {
            a.z[l] = static_cast<const f16*>(grads->z[l]);
            a.dbias[l] = static_cast<f16*>(grads->dbias[l]);
        }
        a.act = grads->act;
    }
    a.partial = static_cast<float*>(partial);
    a.out = (int)out;
    a.op = (int)op;
    a.G = (int)(in / kGroup);
    a.T = (int)batch;
    a.n = L.n;
    a.ip = p.n_cb * kBGroups * kGroup;
    a.n_cb = p.n_cb;
    a.splits = p.splits;
    const int64_t grid = (int64_t)p.n_cb * L.n * p.splits * p.n_tt;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    const hipError_t e = sc.M == 2   ? launch_ct<kScheme2x8>(p.ct, a, (int)grid, stream)
                         : sc.M == 1 ? launch_ct<kScheme1x16>(p.ct, a, (int)grid, stream)
                                     : launch_ct<kSchemeB8M4>(p.ct, a, (int)grid, stream);
    if (e != hipSuccess) return e;
    const Epilogue plain = {{nullptr, nullptr}, nullptr, {nullptr, nullptr}, dx, kActNone};
    return launch_finish(1, a.partial, nullptr, plain, in, a.ip, batch, L.n * p.splits, bias, stream);
}

}  // namespace aqlm
