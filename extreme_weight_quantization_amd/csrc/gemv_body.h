// The decode-phase product's workgroup body (gemv.hip describes it), shared by the plain
// launches of gemv.hip and by those with an epilogue of gemv_act.hip.
//
// KIND kGemvPlain: y = W x, rounded to fp16.
// KIND kGemvAct:   z = W x + bias, y = act(z) + residual (GemvEpi).
// KIND kGemvGated: two layers in one pass.  A tile of 16 matrix-core rows is 8 rows of the
//   gate and the same 8 of the up projection (lanes with l % 16 < 8: gate), so the waves
//   walk ceil(out / 8) tiles exactly as they would walk the 16-row tiles of one layer of
//   2 out rows, x is read once for both, and the thread that adds a gate output's
//   partials also adds its up output's: y = act(zg) zu.  Of the REPL replicas that the LDS
//   codebook holds, half belong to each layer: the replica index of a lane is
//   (layer, l % (REPL / 2)), and with REPL = 8 lane l reads codebook (l / 4) % 2 of its two
//   first, so the 16 lanes served together still touch 16 distinct 16-byte bank groups
//   (2 layers x 2 codebooks x 4 replicas).
// The kinds with an epilogue multiply each codeword of a group with x on its own (two
// products a group for 2x8, four for 4x8) and let the fp32 accumulator add them: the
// matrix cores wait for the lookups anyway, and no sum of codewords is rounded to fp16.
#pragma once
#include "act_math.h"
#include "aqlm_device.h"
#include "aqlm_launch.h"
#include "hidden_pair.h"

namespace aqlm {

// KIND kGemvGatedAt, kGemvPartAt: an expert's products in a mixture-of-experts layer (moe.hip).  Column b of x is row
//   rows.x[b], and results go to row rows.y[b] (GemvRows).  GatedAt writes act(zg) zu as two fp16 numbers (hidden_pair.h), PartAt
//   takes such pairs as columns 2b and 2b + 1 and writes their product in fp32.
enum GemvKind : int { kGemvPlain = 0, kGemvAct = 1, kGemvGated = 2, kGemvGatedAt = 3, kGemvPartAt = 4 };
constexpr bool gemv_gated(int kind) { return kind == kGemvGated || kind == kGemvGatedAt; }
constexpr bool gemv_at(int kind) { return kind == kGemvGatedAt || kind == kGemvPartAt; }

// Rows of the kinds that gather; x and y are in LDS.
struct GemvRows {
    const uint16_t* x;   // rows of x of the columns
    const uint16_t* y;   // rows of the result
    float* part;         // fp32 [..][out] (kGemvPartAt)
};

// What the kinds with an epilogue take next to the first layer's arguments (l = 1: the up
// projection).  residual may be y: each element is read by the thread that then writes it.
struct GemvEpi {
    const uint8_t* codes1;
    const f16* codebooks1;
    const f16* scales1;
    const f16* bias[2];
    const f16* residual;
    f16* z[2];
    int act;
};

// The epilogue of output (b, row), whose products (before the row scales) are p0 and, for
// gated, p1.
template <int KIND>
__device__ __forceinline__ void gemv_finish(float p0, float p1, const f16* __restrict__ scales, f16* y, int b, int row,
                                            int out, const GemvEpi& e) {
    const size_t at = (size_t)b * out + row;
    float z = p0 * (float)scales[row];
    if (e.bias[0] != nullptr) z += (float)e.bias[0][row];
    if (e.z[0] != nullptr) e.z[0][at] = (f16)z;
    float va[1] = {z};
    act_values(e.act, va);
    float v = va[0];
    if constexpr (KIND == kGemvGated) {
        float u = p1 * (float)e.scales1[row];
        if (e.bias[1] != nullptr) u += (float)e.bias[1][row];
        if (e.z[1] != nullptr) e.z[1][at] = (f16)u;
        v *= u;
    } else {
        if (e.residual != nullptr) v += (float)e.residual[at];
    }
    y[at] = (f16)v;
}

// kGemvGatedAt: h = act(zg) zu of (row `at`, `row`), kept as hidden_pair.h says.
__device__ __forceinline__ void gemv_finish_pair(float p0, float p1, const f16* __restrict__ scales, f16* y, int at, int row,
                                                 int out, const GemvEpi& e) {
    float va[1] = {p0 * (float)scales[row]};
    act_values(e.act, va);
    store_pair(va[0] * (p1 * (float)e.scales1[row]), y, at, row, out);
}

constexpr int kGemvWaves = 16;
constexpr int kGemvThreads = kGemvWaves * kWave;
constexpr int kSlabGroups = 32;          // groups per slab (8 products x 4 k-quarters)
constexpr int kRowTile = 16;
// A wave's tile in LDS: row r (output row), column b (batch) at r * 17 + b.  The odd
// stride puts the four k-quarters' writes of one column, and the 16 rows that the
// summing threads read for one column, in distinct bank groups (a stride of 16 made
// both 4-way conflicts).
constexpr int kRedRow = 17;
constexpr int kRedStride = kRowTile * kRedRow;

// How a wave gets the activation operand of a slab (x of 16 batch columns x 32
// groups) into registers:
//   kXDirect      16-byte loads straight into the operand layout;
//   kXStaged8/16  direct-to-LDS loads of the slab's first 8 or 16 batch rows into
//                 a stage of this wave (each 4 consecutive lanes read 64
//                 contiguous bytes of one row), then LDS reads into the operand
//                 layout.
// The operand layout puts a different batch row in each of 16 consecutive
// lanes, so a direct load looks up one cache line per active lane; the staged
// load looks up one per four lanes.
//   kXStaged16in8 16 batch rows through an 8-row stage, in two halves: rows 0-7,
//                 read into the operand layout, then rows 8-15 into the same slots.
//                 Half the LDS of the 16-row stage, so the 2x8 codebooks keep 8
//                 replicas above batch 8, for one more load round trip per slab.
enum XMode : int { kXDirect = 0, kXStaged8 = 1, kXStaged16 = 2, kXStaged16in8 = 3 };
constexpr int kXStageSlots(int xm) {
    return xm == kXStaged16 ? 16 * kSlabGroups : (xm == kXStaged8 || xm == kXStaged16in8) ? 8 * kSlabGroups : 0;
}

// Loads the 8 two-byte codes of a lane's chunk (row, groups g0 .. g0+7),
// packed two per 32-bit word.  The load is unconditional, with the row and
// group indices clamped into the matrix, so that no branch forces an early
// wait on it; groups outside the matrix are masked when they are decoded.
template <bool VEC, int KIND>
__device__ __forceinline__ u32x4 load_codes(const uint8_t* __restrict__ codes, int row, int out,
                                            int g0, int G) {
    const int r = min(row, out - 1);
    if constexpr (!VEC && KIND != kGemvPlain) {
        const size_t total = (size_t)out * G;
        const size_t at = (size_t)r * G + g0;
        if (total >= 8) return settle_codes(load_codes_raw(reinterpret_cast<const uint16_t*>(codes), at, total), at, total);
    }
    const uint16_t* c16 = reinterpret_cast<const uint16_t*>(codes) + (size_t)r * G;
    if constexpr (VEC) {
        // G % 8 == 0: 16-byte aligned chunks; a chunk past the end is clamped to the last one.
        return load_nt16(c16 + min(g0, G - 8));
    } else {
        u32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = (uint32_t)c16[min(g0 + 2 * q, G - 1)] | ((uint32_t)c16[min(g0 + 2 * q + 1, G - 1)] << 16);
        return v;
    }
}

// Group of product q (0..7) in the slab for the lane of k-quarter kq.
__device__ __forceinline__ int slab_group(int kq, int q) { return 8 * kq + q; }

// 16-byte LDS slots of the codebooks of a 2-bit B = 8 scheme with REPL
// replicas: codeword k of codebook m, 8-entry piece h (of H = g / 8) sits in
// slot ((k M + m) H + h) REPL + r (2x8: (2k + m) REPL + r).  1x8 g4 keeps its
// 4-entry codewords in 8-byte slots k REPL + r (half as many 16-byte slots).  4x8 g16 with an
// epilogue: slot ((k H + h) M + m) REPL + r.
// 0 for 1x16.
template <int SCHEME, int REPL>
constexpr int cb_slots() {
    constexpr int M = b8_codebooks(SCHEME);
    return M == 0 ? 0 : M == 1 ? kCodewords2x8 / 2 * REPL : kCodewords2x8 * M * (M / 2) * REPL;
}

// Byte b (0..15) of a lane's 16 bytes of codes.
__device__ __forceinline__ uint32_t code_byte(const u32x4 cv, int b) { return (cv[b >> 2] >> (8 * (b & 3))) & 0xff; }

// Decodes the 8 pieces of 8 inputs that a lane's 16 bytes of codes cover into
// matrix-core A operands (fp16) and accumulates their products with the
// activation operands bx into acc.  Pieces past the end of the row (ok mask
// bit clear) contribute zero.  The lookups of four pieces are issued before
// any of them is used.
//   2x8 (g = 8): piece q is group q, two codewords added in fp16 (exact in
//     fp32, one rounding);
//   1x16: piece q is group q, its codeword gathered from the L2-resident codebook;
//   1x8 g4: piece q is groups 2q and 2q+1, one 8-byte codeword each;
//   4x8 g16 / 8x8 g32: piece q is part q % H of group q / H (H = 2 or 4), the
//     M codewords' parts added in fp32 from codebook 0 upward, rounded once
//     (one piece at a time for 8x8, which would otherwise run out of registers).
// MASKED false: every piece of the chunk is inside the matrix (a whole slab of a
// whole row tile), and ok_mask is not read.
template <int SCHEME, int REPL, bool MASKED, int KIND>
__device__ __forceinline__ f32x4 chunk_mfma(const u32x4 cv, const u32x4* __restrict__ cb_lds,
                                            const f16* __restrict__ codebooks, int rrep,
                                            uint32_t ok_mask, const f16x8 (&bx)[8], f32x4 acc) {
    constexpr int M = b8_codebooks(SCHEME);
    constexpr bool EXACT = KIND != kGemvPlain;   // codewords multiplied one by one
    auto keep = [&](int p) { return !MASKED || ((ok_mask >> p) & 1); };
    if constexpr (M == 1) {
        const u32x2* cb8 = reinterpret_cast<const u32x2*>(cb_lds);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f16x8 a[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int p = 4 * h + q;
                const u32x2 lo = cb8[code_byte(cv, 2 * p) * REPL + rrep];
                const u32x2 hi = cb8[code_byte(cv, 2 * p + 1) * REPL + rrep];
                a[q] = as_f16x8(u32x4{lo[0], lo[1], hi[0], hi[1]});
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a[q] = keep(4 * h + q) ? a[q] : f16x8{};
                acc = mfma16x16x32(a[q], bx[4 * h + q], acc);
            }
        }
        return acc;
    } else if constexpr (M == 4 && EXACT) {
        // 4x8 g16 with an epilogue: lanes take the four codebooks in rotation (which the sum does not
        // feel but in the order of its fp32 additions), so that the 16 lanes served together read 16 distinct bank
        // groups of the half h of a codeword, 4 codebooks x 4 replicas of 16 bytes (in the same
        // order in all lanes: 4-way conflicts, gated 4096x11008 at batch 1 31.4 us).
        const uint32_t lane = threadIdx.x & (kWave - 1);
        const uint32_t rot = lane / (gemv_gated(KIND) ? REPL / 2 : REPL) & 3u;
        uint32_t low[4];   // slot of the i-th codebook's piece 0, codeword 0
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) low[i] = ((rot + i) & 3u) * REPL + rrep;
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
            const uint32_t d = __builtin_amdgcn_alignbit(cv[gi], cv[gi], 8u * rot);
            f16x8 c[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4* at = cb_lds + ((d >> (8 * i)) & 0xffu) * (8 * REPL) + low[i];
                c[0][i] = as_f16x8(at[0]);
                c[1][i] = as_f16x8(at[4 * REPL]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc = mfma16x16x32(keep(2 * gi + h) ? c[h][i] : f16x8{}, bx[2 * gi + h], acc);
        }
        return acc;
    } else if constexpr (M >= 4) {
        constexpr int H = M / 2;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int gi = q / H, h = q % H;
            float sum[8];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const uint32_t k = code_byte(cv, gi * M + m);
                const f16x8 c = as_f16x8(cb_lds[((k * M + m) * H + h) * REPL + rrep]);
#pragma unroll
                for (int t = 0; t < 8; ++t) sum[t] = m == 0 ? (float)c[t] : sum[t] + (float)c[t];
            }
            f16x8 a;
#pragma unroll
            for (int t = 0; t < 8; ++t) a[t] = (f16)sum[t];
            a = keep(q) ? a : f16x8{};
            acc = mfma16x16x32(a, bx[q], acc);
            if constexpr (M == 8) __builtin_amdgcn_sched_barrier(0);
        }
        return acc;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f16x8 a[4];
        if constexpr (SCHEME == kScheme2x8 && REPL == 8) {
            // The two reads of a group take the codebooks in the order (mA, 1 - mA) with
            // mA = (lane / 8) % 2, so the 16 lanes served together read 16 distinct 16-byte
            // bank groups of a 256-byte LDS row (codeword k of codebook m, replica r at byte
            // 256 k + 128 m + 16 r).  v_perm_b32 assembles an address in one instruction:
            // byte 0 from base (16 r + 128 m), byte 1 the code byte, bytes 2-3 zero.  The
            // fp16 sum of the two codewords does not depend on the order of its operands.
            const uint32_t lane = threadIdx.x & (kWave - 1);
            // gated: bit 3 of the lane is the layer, whose replicas are 4 .. 7
            const uint32_t mA = gemv_gated(KIND) ? (lane >> 2) & 1u : (lane >> 3) & 1u;
            const uint32_t r16 = (gemv_gated(KIND) ? (lane & 3u) + 4u * ((lane >> 3) & 1u) : lane & 7u) * 16u;
            const uint32_t base = (r16 + 128u * mA) | ((r16 + 128u * (mA ^ 1u)) << 8);
            const char* cbb = reinterpret_cast<const char*>(cb_lds);
            f16x8 c1[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t d = cv[2 * h + (q >> 1)], hw = 2u * (q & 1);
                const uint32_t ra = __builtin_amdgcn_perm(base, d, 0x0c0c0004u | ((hw + mA) << 8));
                const uint32_t rb = __builtin_amdgcn_perm(base, d, 0x0c0c0005u | ((hw + (mA ^ 1u)) << 8));
                a[q] = as_f16x8(*reinterpret_cast<const u32x4*>(cbb + ra));
                c1[q] = as_f16x8(*reinterpret_cast<const u32x4*>(cbb + rb));
            }
            if constexpr (EXACT) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[q] = keep(4 * h + q) ? a[q] : f16x8{};
                    c1[q] = keep(4 * h + q) ? c1[q] : f16x8{};
                    acc = mfma16x16x32(a[q], bx[4 * h + q], acc);
                    acc = mfma16x16x32(c1[q], bx[4 * h + q], acc);
                }
                continue;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) a[q] = keep(4 * h + q) ? a[q] + c1[q] : f16x8{};
        } else if constexpr (SCHEME == kScheme2x8) {
            static_assert(KIND == kGemvPlain, "the kinds with an epilogue keep 8 replicas");
            f16x8 c1[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t c = (cv[2 * h + (q >> 1)] >> (16 * (q & 1))) & 0xffff;
                a[q] = as_f16x8(cb_lds[(2 * (c & 0xff)) * REPL + rrep]);
                c1[q] = as_f16x8(cb_lds[(2 * (c >> 8) + 1) * REPL + rrep]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) a[q] = keep(4 * h + q) ? a[q] + c1[q] : f16x8{};
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t c = (cv[2 * h + (q >> 1)] >> (16 * (q & 1))) & 0xffff;
                a[q] = as_f16x8(load16(codebooks + (size_t)c * kGroup));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) a[q] = keep(4 * h + q) ? a[q] : f16x8{};
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) acc = mfma16x16x32(a[q], bx[4 * h + q], acc);
    }
    return acc;
}

// The product for one layer, run by workgroup bid of the nwg that serve it.
// XM: how x reaches the registers (XMode).
template <int SCHEME, int REPL, bool VEC, int RTP, int XM, int KIND = kGemvPlain, int TEAM = kGemvWaves>
__device__ __forceinline__ void gemv_body(const uint8_t* __restrict__ codes0, const f16* __restrict__ codebooks0,
                                          const f16* __restrict__ scales, f16* y, const int out,
                                          const int bid, const int nwg, const f16* __restrict__ x, int in, int T,
                                          const GemvEpi epi = {}, const GemvRows rows = {}) {
    constexpr bool GATED = gemv_gated(KIND), AT = gemv_at(KIND);
    constexpr int kTileRows = GATED ? kRowTile / 2 : kRowTile;   // output rows of a tile
    constexpr bool XS = XM == kXStaged8 || XM == kXStaged16 || XM == kXStaged16in8;
    constexpr int kStage = kXStageSlots(XM);    // 16-byte slots of one wave's x stage
    constexpr int kStageRows = kStage / kSlabGroups;
    extern __shared__ u32x4 smem[];
    constexpr int kCbSlots = cb_slots<SCHEME, REPL>();
    // The per-wave partial tiles; with staged x they share the first stages,
    // which are idle whenever the tiles are summed.
    float* red = reinterpret_cast<float*>(smem + kCbSlots);

    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int G = in / kGroup;
    const int n_slab = (G + kSlabGroups - 1) / kSlabGroups;
    const int n_rt = (out + kTileRows - 1) / kTileRows;

    const int lrow = lane & 15;   // A row / B column (batch) of this lane
    const int kq = lane >> 4;     // which 8-group quarter of the slab
    // output row of this lane in a tile, and its layer
    const int trow = GATED ? lrow & 7 : lrow;
    const bool up = GATED && lrow >= 8;
    const uint8_t* codes = up ? epi.codes1 : codes0;
    const f16* codebooks = up ? epi.codebooks1 : codebooks0;
    // codebook replica read by this lane
    const int rrep = GATED ? (REPL / 2) * (int)up + lane % (REPL > 1 ? REPL / 2 : 1) : lane % REPL;
    static_assert(!GATED || SCHEME == kScheme1x16 || REPL % 2 == 0, "replicas of two layers");

    // A team of TEAM waves takes a tile, its waves the tile's slabs in turn.
    constexpr int kTeams = kGemvWaves / TEAM;
    const int team = kTeams == 1 ? 0 : wave / TEAM;
    const int stride = nwg * kTeams;   // between the tiles of a pass

    // First codes and activations of this wave, issued before the codebook is
    // staged so that their memory latency overlaps the LDS fill.
    int rt0 = bid + team * nwg;
    const int s0 = kTeams == 1 ? wave : wave % TEAM;
    u32x4 cnext[RTP];
#pragma unroll
    for (int i = 0; i < RTP; ++i) {
        const int rt = rt0 + i * stride;
        cnext[i] = (s0 < n_slab && rt < n_rt)
                       ? load_codes<VEC, KIND>(codes, rt * kTileRows + trow, out, s0 * kSlabGroups + kq * 8, G)
                       : u32x4{0u, 0u, 0u, 0u};
    }
    f16x8 bx[8];
    auto load_x = [&](int s) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int grp = s * kSlabGroups + slab_group(kq, q);
            bx[q] = (lrow < T && grp < G)
                        ? as_f16x8(load16(x + (size_t)(AT ? (int)rows.x[lrow] : lrow) * in + (size_t)grp * kGroup))
                        : f16x8{};
        }
    };
    // Staged x: batch row b, group c of the slab sits in slot kSlabGroups * b + (c ^ b)
    // of the wave's stage, so the 16 lanes that read one group for 16 rows hit 16
    // distinct bank groups.  Load i fills slots 64 i .. 64 i + 63 (rows 2i, 2i + 1)
    // and is issued only if row 2i is in the batch; a row 2i + 1 past the batch
    // repeats row 2i, a group past the matrix the row's last group.  Every read
    // stays in x.  Stage rows past the batch keep stale values: a matrix-core
    // column depends on its own B column only, and the columns past the batch
    // are discarded; groups past the matrix are zeroed when read.
    u32x4* const xst = smem + kCbSlots + (XS ? wave * kStage : 0);
    // Batch rows r0 .. r0 + kStageRows - 1 of slab s into the stage (stage row b holds
    // batch row r0 + b).
    auto stage_rows = [&](int s, int r0) {
        // The lane index passes through an empty asm statement so that the
        // address arithmetic stays here instead of being hoisted out of the
        // loops as eight live 64-bit pointers.
        int l = lane;
        asm volatile("" : "+v"(l));
#pragma unroll
        for (int i = 0; i < kStageRows / 2; ++i) {
            if (r0 + 2 * i >= T) break;   // rows past the batch only feed discarded columns
            const int b = 2 * i + (l >> 5);
            const int grp = min(s * kSlabGroups + ((l & 31) ^ b), G - 1);
            const int row = AT ? (int)rows.x[min(r0 + b, T - 1)] : min(r0 + b, T - 1);
            __builtin_amdgcn_global_load_lds(
                (const void*)(x + (size_t)row * in + (size_t)grp * kGroup),
                lds_ptr(xst + 64 * i), 16, 0, 0);
        }
    };
    auto stage_x = [&](int s) { stage_rows(s, 0); };
    // Waits for every load of this wave (the stage among them), reads the operand
    // layout; groups past the end of the row read as zero so that their
    // products stay zero whatever x holds.
    auto read_x = [&](int s) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
        asm volatile("" ::: "memory");
        const int b = lrow & (kStageRows - 1);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int c = slab_group(kq, q);
            const f16x8 v = as_f16x8(xst[kSlabGroups * b + (c ^ b)]);
            bx[q] = (s * kSlabGroups + c < G) ? v : f16x8{};
        }
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);   // the stage is free again
        asm volatile("" ::: "memory");
        if constexpr (XM == kXStaged16in8) {
            // the second half: rows 8-15 into the same slots, read by the lanes of
            // operand columns 8-15
            if (T > kStageRows) {
                __builtin_amdgcn_sched_barrier(0);
                stage_rows(s, kStageRows);
                asm volatile("" ::: "memory");
                __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
                asm volatile("" ::: "memory");
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int c = slab_group(kq, q);
                    const f16x8 v = as_f16x8(xst[kSlabGroups * b + (c ^ b)]);
                    if (lrow >= kStageRows) bx[q] = (s * kSlabGroups + c < G) ? v : f16x8{};
                }
                __builtin_amdgcn_s_waitcnt(kWaitLgkm0);   // the stage is free again
                asm volatile("" ::: "memory");
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    int s_loaded = -1;   // slab whose activations are in bx
    if constexpr (XS) {
        if (s0 < n_slab) stage_x(s0);
    } else {
        load_x(s0);
        s_loaded = s0;
    }

    // 1x16: warm this XCD's L2 with a 32 KB slice of the codebook (workgroups
    // are dealt to the 8 XCDs round-robin, so 32 consecutive workgroups of one
    // XCD cover the whole 1 MiB); the gathers that follow then hit in L2.
    u32x4 warm = {0u, 0u, 0u, 0u};
    if constexpr (SCHEME == kScheme1x16) {
        const size_t slice = (size_t)((blockIdx.x >> 3) & 31) * (32768 / 16);
        const u32x4* cb16 = reinterpret_cast<const u32x4*>(codebooks0);
        warm = load16(cb16 + slice + tid) ^ load16(cb16 + slice + kGemvThreads + tid);
        if constexpr (GATED) {
            const u32x4* cb16u = reinterpret_cast<const u32x4*>(epi.codebooks1);
            warm ^= load16(cb16u + slice + tid) ^ load16(cb16u + slice + kGemvThreads + tid);
        }
    }

    constexpr int kM = b8_codebooks(SCHEME);
    if constexpr (kM == 1) {
        // 8-byte slot j = k * REPL + r holds codeword k (4 fp16); loads first, then LDS writes
        constexpr int kSlots8 = 2 * kCbSlots;
        constexpr int kFill = (kSlots8 + kGemvThreads - 1) / kGemvThreads;
        u32x2* cb8 = reinterpret_cast<u32x2*>(smem);
        u32x2 fv[kFill];
#pragma unroll
        for (int it = 0; it < kFill; ++it) {
            const int j = min(it * kGemvThreads + tid, kSlots8 - 1);
            const f16* cbl = GATED && j % REPL >= REPL / 2 ? epi.codebooks1 : codebooks0;
            fv[it] = *reinterpret_cast<const u32x2*>(cbl + (size_t)(j / REPL) * 4);
        }
#pragma unroll
        for (int it = 0; it < kFill; ++it) {
            const int j = it * kGemvThreads + tid;
            if (j < kSlots8) cb8[j] = fv[it];
        }
    } else if constexpr (kM >= 2) {
        // Slot j holds piece h of codeword k of codebook m, replica r:
        // j = ((k M + m) H + h) REPL + r.  Direct-to-LDS loads: load it of wave w fills
        // slots it * 1024 + 64 w .. + 63, lane l slot it * 1024 + 64 w + l, from the 16 B
        // of its piece; then every load of the wave is waited for (the code and x
        // loads issued before it too).
        constexpr int kH = kM / 2, kG = 4 * kM;
        static_assert(kCbSlots % kGemvThreads == 0, "whole waves of slots");
#pragma unroll
        for (int it = 0; it < kCbSlots / kGemvThreads; ++it) {
            const int j = it * kGemvThreads + tid;
            const int kmh = j / REPL;
            const int km = kM == 4 && KIND != kGemvPlain ? kmh / 8 * 4 + kmh % 4 : kmh / kH;
            const int h = kM == 4 && KIND != kGemvPlain ? kmh / 4 % 2 : kmh % kH;
            const f16* cbl = GATED && j % REPL >= REPL / 2 ? epi.codebooks1 : codebooks0;
            __builtin_amdgcn_global_load_lds(
                (const void*)(cbl + (size_t)((km % kM) * kCodewords2x8 + km / kM) * kG + h * 8),
                lds_ptr(smem + it * kGemvThreads + wave * 64), 16, 0, 0);
        }
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
    }
    __syncthreads();

    for (; rt0 - team * nwg < n_rt; rt0 += stride * RTP) {
        f32x4 acc[RTP];
#pragma unroll
        for (int i = 0; i < RTP; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};

        for (int s = s0; s < n_slab; s += TEAM) {
            u32x4 ccur[RTP];
#pragma unroll
            for (int i = 0; i < RTP; ++i) ccur[i] = cnext[i];
            if constexpr (XS) {
                if (s != s_loaded) {
                    if (s_loaded >= 0) stage_x(s);   // the first slab was staged before the codebook
                    read_x(s);
                    s_loaded = s;
                }
            }
            // Prefetch the codes of this wave's next slab (or of the next pass).
            {
                int sn = s + TEAM, rtn = rt0;
                if (sn >= n_slab) { sn = s0; rtn = rt0 + stride * RTP; }
#pragma unroll
                for (int i = 0; i < RTP; ++i) {
                    const int rt = rtn + i * stride;
                    cnext[i] = (sn < n_slab && rt < n_rt)
                                   ? load_codes<VEC, KIND>(codes, rt * kTileRows + trow, out, sn * kSlabGroups + kq * 8, G)
                                   : u32x4{0u, 0u, 0u, 0u};
                }
            }
            if constexpr (!XS) {
                if (s != s_loaded) { load_x(s); s_loaded = s; }
            }
            uint32_t gmask = 0u;   // bit q: the group of product q is inside the row
#pragma unroll
            for (int q = 0; q < 8; ++q)
                gmask |= (s * kSlabGroups + slab_group(kq, q) < G) ? (1u << q) : 0u;
            const bool whole_slab = (s + 1) * kSlabGroups <= G;   // uniform over the wave
#pragma unroll
            for (int i = 0; i < RTP; ++i) {
                const int rt = rt0 + i * stride;
                if (rt >= n_rt) break;
                if (whole_slab && (rt + 1) * kTileRows <= out) {
                    acc[i] = chunk_mfma<SCHEME, REPL, false, KIND>(ccur[i], smem, codebooks, rrep, 0u, bx, acc[i]);
                } else {
                    const uint32_t ok = (rt * kTileRows + trow < out) ? gmask : 0u;
                    acc[i] = chunk_mfma<SCHEME, REPL, true, KIND>(ccur[i], smem, codebooks, rrep, ok, bx, acc[i]);
                }
            }
        }

        // Sum the per-wave partial tiles, scale, round to fp16.
#pragma unroll
        for (int i = 0; i < RTP; ++i) {
            if (rt0 - team * nwg + i * stride >= n_rt) break;   // no team has a tile
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave * kRedStride + (4 * kq + r) * kRedRow + lrow] = acc[i][r];
            __syncthreads();
            static_assert(kTeams * kTileRows * 16 <= kGemvThreads, "a thread an element of the teams' tiles");
            if (tid < kTeams * kTileRows * 16) {
                const int tm = kTeams == 1 ? 0 : tid / (kTileRows * 16), w0 = tm * TEAM;   // the element's team and its first wave
                const int rt = rt0 + (tm - team) * nwg + i * stride;
                const int b = kTeams == 1 ? tid / kTileRows : tid / kTileRows % 16, rr = tid % kTileRows;
                const int row = rt * kTileRows + rr;
                if constexpr (KIND == kGemvPartAt) {
                    if (2 * b < T && row < out) {   // T is even
                        float sum = 0.f;
#pragma unroll
                        for (int w = w0; w < w0 + TEAM; ++w)
                            sum += red[w * kRedStride + rr * kRedRow + 2 * b] +
                                   red[w * kRedStride + rr * kRedRow + 2 * b + 1] * (1.f / kPairFine);
                        rows.part[(size_t)rows.y[b] * out + row] = sum * kPairUnit * (float)scales[row];
                    }
                } else if (b < T && row < out) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = w0; w < w0 + TEAM; ++w) sum += red[w * kRedStride + rr * kRedRow + b];
                    if constexpr (KIND == kGemvPlain) {
                        y[(size_t)b * out + row] = (f16)(sum * (float)scales[row]);
                    } else {
                        float sum1 = 0.f;
                        if constexpr (GATED) {
#pragma unroll
                            for (int w = w0; w < w0 + TEAM; ++w) sum1 += red[w * kRedStride + (8 + rr) * kRedRow + b];
                        }
                        if constexpr (AT) gemv_finish_pair(sum, sum1, scales, y, rows.y[b], row, out, epi);
                        else gemv_finish<KIND>(sum, sum1, scales, y, b, row, out, epi);
                    }
                }
            }
        }
        // Staged x, several slabs per wave: the next pass stages its first slab
        // over the tiles just summed.
        if constexpr (XS) {
            if (n_slab > TEAM) __syncthreads();
        }
    }
    // Keeps the L2 warm-up loads alive; the condition never holds (tid < 1024).
    if ((warm[0] ^ warm[3]) == 0x9e3779b9u && tid == 0xffff) y[0] = (f16)0.f;
}

}  // namespace aqlm
