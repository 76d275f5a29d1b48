// Products of a small batch (tens to hundreds of tokens) straight from the codes, 2x8, 1x16 and
// 4x8 g16:
//   P_l[t][i] = sum_k Wc_l[i][k] x[t][k]  for one layer, or the gate and up projections,
// then the epilogue of act_launch.h.
//
// "The AQLM Quantization Algorithm, Explained", Figure 2 of the MCQ section (a group's
// weights are the sum of one codeword per codebook, times the row's scale) and section
// "Key AQLM quantization parameters" (2x8 and 1x16 at g = 8, 4x8 at g = 16).
//
// Between the decode-phase product (one 16-column matrix-core tile of tokens) and prefill (where decoding
// the weights once into memory pays) a call is bound by its codeword lookups, the matrix
// cores and fixed latencies.  So the weights never leave the registers they are looked up into:
//
//  * the matrix-core operand of W wants lane l to hold 8 consecutive inputs of row l % 16,
//    which is one group of 8: a lane looks its groups up (2x8: two codewords from the LDS
//    copy of the codebooks, 8 replicas, conflict-free as in gemv.hip; 1x16: one 16-byte
//    gather from L2, half a step ahead; 4x8 g16: the halves of four codewords from 2 replicas,
//    2-way conflicts) and multiplies each codeword on its own, so no weight is rounded.  Their sums
//    in fp16 would halve the products, for one rounding of every weight (2x8; two of 4x8 g16's pairs): gated
//    4096x11008 at 256 tokens 97 -> 81 us, at 1000x2733 and 130 16.9 -> 16.3, 4x8 g16 at 40 46 -> 38;
//  * a workgroup of 16 waves covers 256 rows (gated: 8 gate and 8 up rows a wave) and
//    walks slabs of 32 groups (256 inputs); the x tile of a slab, BM tokens, sits in LDS
//    for all waves, three stages of direct-to-LDS loads, one barrier a slab;
//  * the (token tile, row block, slab) units are dealt to one workgroup per CU in equal
//    contiguous runs, so every CU has the same work whatever the shape; each run's part of
//    a row block is written as fp32 partial sums, and skinny_finish_kernel adds a
//    block's parts in order, applies the row scale and the epilogue, and rounds once.
//
// What bounds it.  1x16: the gathers, one L2 request each; 4096x11008 at 48 tokens, main kernel
// 34 us by the profiler for 5.6 M of them, 170 G/s of the 264 G/s that a kernel of nothing
// else reaches (runs of 3 units where 2.7 would be even, and about 8 us to start and end).
// 2x8 and 4x8 g16: matrix cores and LDS reads alike (gated 4096x11008 2x8 at 256 tokens: 5.6 M products of 16
// cycles and 2.8 M reads at 8 clocks each are 50 % each of the kernel's 85 us at 2.1 GHz), at small sizes the
// start, two dependent loads and the end of a run.
//
// LDS layout of an x stage: token b, group c in 16-byte slot 32 b + (x_place(c) ^ (b % 16)).
// A 16-byte LDS read serves 16 lanes at a time: 0-3, 12-15 and 20-27; 4-11, 16-19 and 28-31;
// likewise above 32.  Lanes 0-15 read group q and lanes 16-31 group 8 + q of 16 tokens, and
// x_place makes those two differ in bits 2 and 3 of the slot, so that the 16 bank groups are distinct
// (with c itself there, bit 3 alone, every read was a 2-way conflict).
#include <algorithm>
#include <type_traits>

#include "act_bias.h"
#include "act_launch.h"
#include "act_math.h"
#include "aqlm_device.h"

namespace aqlm {

namespace {

constexpr int kKTiles = 16;                                  // matrix-core row tiles of a workgroup (256 rows)
constexpr int kKSlab = 32;                                  // groups per step
// Steps of x (LDS stages) and codes (registers) in flight: what 160 KB of LDS hold (1x16 at 128
// tokens: two stages of 64 KB; its steps are long enough for one step ahead).
constexpr int skinny_stages(int bm) { return bm == 128 ? 2 : 3; }
constexpr int kKRepl = 8;                                   // 2x8 codebook replicas in LDS
constexpr int kKCbBytes = 2 * kCodewords2x8 * kKRepl * 16;   // 64 KB; 4x8 g16: two replicas
constexpr bool lds_codebooks(int scheme) { return scheme != kScheme1x16; }
// The kernels that have a short form for a last token tile that is at most half full.  Not 1x16: its
// gathers, which bound it, stay the same.
constexpr bool skinny_halves(int scheme, int bm) { return bm == 64 && lds_codebooks(scheme); }

// Units dealt to W workgroups in contiguous runs.  A unit takes one place; or (`full` >= 0, for a
// last token tile at most half full) the units of the other tiles, the first `full`, take two,
// and those of the last tile, which multiply half the columns, one.  The
// `places` go to the workgroups in intervals of q or q + 1 (places = q W + r): that of w begins at
// floor(w places / W) = w q + floor(w r / W), and a unit belongs to the interval that its first
// place is in.  W <= kSkinnyWorkgroups, so w r fits 32 bits; q >= 2 with `full`, so that no run is
// empty.
struct Runs {
    int places, W, q, r, full;
};
__device__ __forceinline__ int run_place(int w, const Runs& v) { return w * v.q + (int)((uint32_t)(w * v.r) / (uint32_t)v.W); }
// The first unit of run w: the first whose place is at or after the interval's begin.
__device__ __forceinline__ int run_begin(int w, const Runs& v) {
    const int p = run_place(w, v);
    if (v.full < 0) return p;
    return p <= 2 * v.full ? (p + 1) >> 1 : p - v.full;
}
// The workgroup whose run holds unit u: an estimate within one (fewer than 2^30 places: a float
// quotient times at most 256 is off by far less), then exact.
__device__ __forceinline__ int run_of(int u, const Runs& v) {
    const int p = v.full < 0 ? u : u + min(u, v.full);
    int w = min((int)((float)p * ((float)v.W / (float)v.places)), v.W - 1);
    if (run_place(w, v) > p) --w;
    if (w + 1 < v.W && run_place(w + 1, v) <= p) ++w;
    return w;
}

// Place of group c in a row of the x stage (its own inverse): bit 2 flipped by bit 3.
__device__ __forceinline__ int x_place(int c) { return c ^ (c >> 1 & 4); }

struct SkinnyArgs {
    const uint8_t* codes[2];
    const f16* codebooks[2];
    const f16* x;
    float* partial;   // [slot][t][l][op]
    int out, op, G, T;
    int n_slab, n_blk;   // slabs of a row; row blocks
    int half_tile;       // the token tile that is at most half full, or -1
    Runs runs;           // of token tiles x row blocks x slabs
};

// 16 bytes of the workgroup's LDS (dynamic only, so it starts at address 0).
__device__ __forceinline__ u32x4 lds16(uint32_t byte) {
    return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>((uintptr_t)byte);
}

// How a row divides into slabs and 16-byte pieces of codes: whole slabs (in % 256 == 0), whole
// pieces (in % 64 == 0), or neither.
enum RowKind : int { kRowWhole = 0, kRowVec = 1, kRowAny = 2 };

// Zeros that the direct-to-LDS loads of x read in the place of groups past the row.
__device__ const u32x4 skinny_zero = {0u, 0u, 0u, 0u};

// RT: row tiles of a wave (16 / RT waves a workgroup).
template <int SCHEME, int BM, bool GATED, int ROW, int RT>
__global__ __launch_bounds__(64 * kKTiles / RT) __attribute__((amdgpu_waves_per_eu(4 / RT, 4 / RT))) void skinny_kernel(
    const SkinnyArgs a) {
    extern __shared__ u32x4 smem[];
    constexpr int kThreads = 64 * kKTiles / RT;
    constexpr int kCT = BM / 16;                              // column tiles of tokens
    constexpr int kXStage = BM * kKSlab;                      // 16-byte slots of a stage
    constexpr int kNX = kXStage / kThreads;                   // x loads a wave issues a step
    constexpr int kR = skinny_stages(BM);                     // steps of x and of codes in flight
    constexpr bool kRagged = ROW != kRowWhole;                // the last slab may have groups past the row
    constexpr bool kCbLds = lds_codebooks(SCHEME), kFour = SCHEME == kSchemeB8M4;
    constexpr uint32_t kXOff = kCbLds ? kKCbBytes : 0;
    // vector loads that every step issues after the x tile that its end waits for: with three
    // stages (that tile: a step ago) all of its own, the x tile, the codes, the gathers; with two, the codes and half the gathers
    constexpr int kGathers = SCHEME == kScheme1x16 ? 4 * RT : 0;   // of half a step
    constexpr int kIssued = kR == 2 ? RT + kGathers : kNX + RT + 2 * kGathers;
    constexpr int kTileRows = GATED ? 8 : 16;
    constexpr int kN = GATED ? 2 : 1;
    constexpr bool kHalves = skinny_halves(SCHEME, BM);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lrow = lane & 15, kq = lane >> 4;
    const bool up = GATED && lrow >= 8;
    const int trow = GATED ? lrow & 7 : lrow;
    const uint16_t* codes = reinterpret_cast<const uint16_t*>(up ? a.codes[1] : a.codes[0]);
    const f16* codebooks = up ? a.codebooks[1] : a.codebooks[0];
    const int G = a.G, n_slab = a.n_slab;
    const int wid = xcd_run((int)blockIdx.x, (int)gridDim.x);
    const int u0 = run_begin(wid, a.runs), n = run_begin(wid + 1, a.runs) - u0;   // n >= 1

    // a unit is (token tile t, row block b, slab s), s fastest
    struct Unit { int t, b, s; };
    auto next = [&](Unit& v) {
        const bool row = v.s == n_slab - 1, col = row && v.b == a.n_blk - 1;
        v.s = row ? 0 : v.s + 1;
        v.b = col ? 0 : v.b + (row ? 1 : 0);
        v.t += col ? 1 : 0;
    };
    // the unit of step `at`
    struct Ahead { Unit v; int at; };
    auto advance = [&](Ahead& p) {
        next(p.v);
        ++p.at;
    };
    // the 8 codes of this lane in a unit: rows past the layer repeat its last row (their
    // outputs are not used), groups past the row its last 8 (masked when used); kRowAny: as
    // loaded, settle_codes puts them in place when they are used
    auto codes_at = [&](const Unit& v, int rt) -> size_t {
        const int row = min((v.b * kKTiles + wave * RT + rt) * kTileRows + trow, a.out - 1);
        const int g0 = v.s * kKSlab + 8 * kq;
        return (size_t)row * G + (ROW != kRowAny ? min(g0, G - 8) : g0);
    };
    auto load_codes = [&](const Unit& v, int rt) -> u32x4 {
        if constexpr (ROW != kRowAny) return load_nt16(codes + codes_at(v, rt));
        return load_codes_raw(codes, codes_at(v, rt), (size_t)a.out * G);
    };
    auto settle = [&](const u32x4 (&c)[RT], const Unit& v, u32x4 (&o)[RT]) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            o[rt] = ROW == kRowAny ? settle_codes(c[rt], codes_at(v, rt), (size_t)a.out * G) : c[rt];
    };
    // x of a unit into a stage: load i of a wave fills slots 64 (wave kNX + i) .. + 63, two tokens;
    // tokens past the batch repeat its last one, groups past the row are zero
    auto load_x = [&](const Unit& v, int stage) {
        u32x4* dst = smem + kXOff / 16 + stage * kXStage;
#pragma unroll
        for (int i = 0; i < kNX; ++i) {
            const int slot = 64 * (wave * kNX + i) + lane;
            const int b = slot / kKSlab, c = x_place(slot % kKSlab ^ (b & 15));
            const int tok = min(v.t * BM + b, a.T - 1), grp = v.s * kKSlab + c;
            const f16* src = a.x + ((size_t)tok * G + grp) * kGroup;
            if constexpr (kRagged) src = grp < G ? src : reinterpret_cast<const f16*>(&skinny_zero);
            __builtin_amdgcn_global_load_lds((const void*)src, lds_ptr(dst + 64 * (wave * kNX + i)), 16, 0, 0);
        }
    };
    // 1x16: the codewords of half h (four groups) of a unit's codes
    auto gather = [&](const u32x4 (&cv)[RT], int h, u32x4 (&e)[RT][4]) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                e[rt][q] =
                    load16(codebooks + (size_t)((cv[rt][2 * h + (q >> 1)] >> (16 * (q & 1))) & 0xffffu) * kGroup);
    };

    if constexpr (kCbLds) {
        // 2x8: slot (2 k + m) 8 + r, codeword k of codebook m (gated: the gate's for r < 4);
        // 4x8 g16: slot 16 k + 8 h + 2 m + r, half h of it (gated: the gate's for r = 0)
#pragma unroll
        for (int it = 0; it < kKCbBytes / 16 / kThreads; ++it) {
            const int slot = it * kThreads + tid;
            const f16* cbl = GATED && (tid & (kFour ? 1 : 4)) != 0 ? a.codebooks[1] : a.codebooks[0];
            const f16* src = kFour ? cbl + (size_t)((slot >> 1 & 3) * kCodewords2x8 + (slot >> 4)) * 16 + (slot >> 3 & 1) * 8
                                   : cbl + (size_t)((slot >> 3 & 1) * kCodewords2x8 + (slot >> 4)) * kGroup;
            __builtin_amdgcn_global_load_lds((const void*)src, lds_ptr(smem + it * kThreads + wave * kWave), 16, 0, 0);
        }
    }
    const int blk0 = (int)((uint32_t)u0 / (uint32_t)n_slab), tile0 = (int)((uint32_t)blk0 / (uint32_t)a.n_blk);
    Unit cur{tile0, blk0 - tile0 * a.n_blk, u0 - blk0 * n_slab};   // the unit multiplied
    Ahead px{cur, 0}, pc{cur, 0};                                  // the next x tile and codes to load
    u32x4 ring[kR][RT];   // codes of step k in ring[k % kR]
    auto load_ring = [&](u32x4 (&r)[RT]) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) r[rt] = load_codes(pc.v, rt);
        advance(pc);
    };
#pragma unroll
    for (int d = 0; d < kR; ++d) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) ring[d][rt] = u32x4{0u, 0u, 0u, 0u};
        if (d < n) load_ring(ring[d]);
    }
#pragma unroll
    for (int d = 0; d < kR - 1; ++d) {
        if (d < n) {
            load_x(px.v, d);
            advance(px);
        }
    }
    u32x4 e[2][RT][4] = {};   // 1x16: codewords of the two halves of a step, gathered half a step ahead
    if constexpr (SCHEME == kScheme1x16) {
        u32x4 c[RT];
        settle(ring[0], cur, c);
        gather(c, 0, e[0]);
    }
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
    __syncthreads();

    const uint32_t mA = GATED ? (lane >> 2) & 1u : (lane >> 3) & 1u;
    const uint32_t r16 = (GATED ? (lane & 3u) + 4u * (uint32_t)up : lane & 7u) * 16u;
    const uint32_t base = (r16 + 128u * mA) | ((r16 + 128u * (mA ^ 1u)) << 8);
    // 4x8 g16: lane l looks up codebooks l, l + 1, .. (mod 4) in turn, so that 16 lanes hit 8 of
    // the 16 bank groups twice; byte i: the slot of its i-th codebook in a codeword's 256 bytes
    const uint32_t rot = lane & 3u, rep = 16u * (GATED ? (uint32_t)up : (lane >> 2) & 1u);
    const uint32_t base4 = (32u * rot + rep) | ((32u * ((rot + 1u) & 3u) + rep) << 8) |
                           ((32u * ((rot + 2u) & 3u) + rep) << 16) | ((32u * ((rot + 3u) & 3u) + rep) << 24);
    const uint32_t xlane = kXOff + 16u * (uint32_t)(kKSlab * lrow + (x_place(8 * kq) ^ lrow));
    f32x4 acc[RT][kCT];
    auto clear = [&]() {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int j = 0; j < kCT; ++j) acc[rt][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    clear();

    // the products of one unit; xs: this lane's place in the stage, left: its groups inside
    // the row (those past it count as zero: x is zero there, W is made so).  The LDS reads of
    // group q + 1 are spread between the products of group q, so that both units stay busy
    // (all reads of a half first: the step took the sum of both, 7300 clocks for 64 tokens).
    constexpr int kLook = kFour ? 4 : 2;   // codewords of a weight
    auto fetch = [&](const u32x4 (&cv)[RT], uint32_t xs, int q, f16x8 (&w)[RT][kLook], auto& xv) {
        constexpr int kC = std::extent_v<std::remove_reference_t<decltype(xv)>>;
        if constexpr (kFour) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint32_t d = __builtin_amdgcn_alignbit(cv[rt][q >> 1], cv[rt][q >> 1], 8u * rot);
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    w[rt][i] = as_f16x8(lds16(__builtin_amdgcn_perm(base4, d, 0x0c0c0004u + i + (i << 8)) + 128u * (q & 1)));
            }
        } else if constexpr (SCHEME == kScheme2x8) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint32_t d = cv[rt][q >> 1], hw = 2u * (q & 1);
                w[rt][0] = as_f16x8(lds16(__builtin_amdgcn_perm(base, d, 0x0c0c0004u | ((hw + mA) << 8))));
                w[rt][1] = as_f16x8(lds16(__builtin_amdgcn_perm(base, d, 0x0c0c0005u | ((hw + (mA ^ 1u)) << 8))));
            }
        }
        const uint32_t xa = xs ^ (uint32_t)(q << 4);
#pragma unroll
        for (int j = 0; j < kC; ++j) xv[j] = as_f16x8(lds16(xa + (uint32_t)(j * 16 * kKSlab * 16)));
    };
    auto multiply = [&](auto columns, const u32x4 (&cv)[RT], u32x4 (&e)[2][RT][4], const u32x4 (&ahead)[RT], bool more,
                        uint32_t xs, int left) {
        constexpr int kC = decltype(columns)::value;   // column tiles multiplied
        constexpr int kReads = kC + (kCbLds ? kLook * RT : 0), kProducts = RT * kC * (kCbLds ? kLook : 1);
        f16x8 w[2][RT][kLook], xv[2][kC];
        fetch(cv, xs, 0, w[0], xv[0]);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q + 1 < 8) fetch(cv, xs, q + 1, w[(q + 1) & 1], xv[(q + 1) & 1]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                // every codeword on its own: no sum of them is rounded
                constexpr int kEach = kCbLds ? kLook : 1;
#pragma unroll
                for (int m = 0; m < kEach; ++m) {
                    f16x8 c = w[q & 1][rt][m];
                    if constexpr (!kCbLds) c = as_f16x8(e[q >> 2][rt][q & 3]);
                    if constexpr (kRagged) c = q < left ? c : f16x8{};
#pragma unroll
                    for (int j = 0; j < kC; ++j) acc[rt][j] = mfma16x16x32(c, xv[q & 1][j], acc[rt][j]);
                }
            }
            if (q + 1 < 8) {
#pragma unroll
                for (int i = 0; i < (kReads < kProducts ? kReads : kProducts); ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one matrix product
                    __builtin_amdgcn_sched_group_barrier(0x100, kReads <= kProducts ? 1 : (kReads + kProducts - 1) / kProducts, 0);   // LDS reads
                }
                if constexpr (kReads < kProducts) __builtin_amdgcn_sched_group_barrier(0x008, kProducts - kReads, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (!kCbLds) {
                if (q == 3 && more) gather(ahead, 0, e[0]);   // the first half of the next step's codewords
            }
        }
    };
    // the run's part of a row block: lane holds rows 4 kq + r of token l % 16 of each column tile
    auto flush = [&](const Unit& v) {
        const int first = run_of((v.t * a.n_blk + v.b) * n_slab, a.runs);
        const int l = GATED ? kq >> 1 : 0;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int tile0 = (v.b * kKTiles + wave * RT + rt) * kTileRows;
            const int r0 = tile0 + (GATED ? 4 * (kq & 1) : 4 * kq);
            if (tile0 >= a.op) break;
#pragma unroll
            for (int j = 0; j < kCT; ++j) {
                const int tok = v.t * BM + 16 * j + lrow;
                if (tok < a.T)
                    *reinterpret_cast<f32x4*>(a.partial + (((size_t)(wid - first) * a.T + tok) * kN + l) * a.op + r0) =
                        acc[rt][j];
            }
        }
        clear();
    };

    // Step k: stage and ring slot are fixed in the unrolled round, each register redefined
    // after its last use, so no wait but for what is used next.  Nothing is loaded past the last unit.
    for (int k0 = 0; k0 < n; k0 += kR) {
#pragma unroll
        for (int d = 0; d < kR; ++d) {
            const int k = k0 + d;
            if (d > 0 && k >= n) break;
            // the address arithmetic stays in the step (hoisted, it would hold 24 registers)
            uint32_t xs = xlane + (uint32_t)(d * kXStage * 16);
            asm volatile("" : "+v"(xs));
            u32x4 c[RT], ahead[RT];
            settle(ring[d], cur, c);
            Unit after = cur;
            next(after);
            if constexpr (SCHEME == kScheme1x16) {
                settle(ring[(d + 1) % kR], after, ahead);
                gather(c, 1, e[1]);
            }
            if (px.at < n) {
                load_x(px.v, (d + kR - 1) % kR);   // this stage was read last in step k - 1
                advance(px);
            }
            __builtin_amdgcn_sched_barrier(0);
            const int left = G - cur.s * kKSlab - 8 * kq;
            using All = std::integral_constant<int, kCT>;
            if constexpr (kHalves) {
                using Half = std::integral_constant<int, kCT / 2>;
                if (cur.t == a.half_tile) multiply(Half{}, c, e, ahead, k + 1 < n, xs, left);
                else multiply(All{}, c, e, ahead, k + 1 < n, xs, left);
            } else {
                multiply(All{}, c, e, ahead, k + 1 < n, xs, left);
            }
            if (pc.at < n) load_ring(ring[d]);
            if (after.s == 0 || k == n - 1) flush(cur);
            cur = after;
            if (k + 1 < n) {
                // x of step k + 1 has landed: the kIssued newest loads are later ones, where all
                // of this step's were issued; near the end everything is waited for
                __builtin_amdgcn_sched_barrier(0);
                asm volatile("" ::: "memory");
                if (k + kR < n) __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kIssued < 16 ? kIssued : 15));
                else __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
}

struct FinishArgs {
    const float* partial;
    const f16* scales[2];
    const f16* bias[2];
    const f16* residual;   // may be y
    f16* z[2];
    f16* y;
    const float* units;    // factors of the tokens' sums, or NULL
    int out, op, T, act;
    int parts;      // > 0: everywhere; else the runs that share the output's row block
    int bm, blk_rows, n_slab, n_blk;
    Runs runs;
    int blocks;     // workgroups of the outputs; those after them add bias sums
    BiasSum sums;
};

// Adds `parts` parts of 4 outputs of N layers in order, kAhead of them in flight; one past the last
// repeats it and is not added.
template <int N, int kAhead>
__device__ __forceinline__ void add_parts(const float* p, size_t step, int op, int parts, f32x4 (&sum)[N]) {
    for (int s0 = 0; s0 < parts; s0 += kAhead, p += kAhead * step) {
        f32x4 v[kAhead][N];
#pragma unroll
        for (int s = 0; s < kAhead; ++s)
#pragma unroll
            for (int l = 0; l < N; ++l)
                v[s][l] = *reinterpret_cast<const f32x4*>(p + (size_t)min(s, parts - 1 - s0) * step + (size_t)l * op);
#pragma unroll
        for (int s = 0; s < kAhead; ++s)
#pragma unroll
            for (int l = 0; l < N; ++l)
#pragma unroll
                for (int r = 0; r < 4; ++r) sum[l][r] += s0 + s < parts ? v[s][l][r] : 0.f;
    }
}

// Thread: 4 outputs of a token.  The parts of its row block are the runs from the one that
// holds the block's first unit to the one that holds its last, added in that order.
template <int N>
__global__ __launch_bounds__(256) void skinny_finish_kernel(const FinishArgs a) {
    if ((int)blockIdx.x >= a.blocks) {
        bias_sum_block(a.sums, (int)blockIdx.x - a.blocks);
        return;
    }
    const int per = a.op / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.T * per) return;
    // the quotient of a product below 2^31 in 32 bits (a 64-bit one costs more than the rest of the thread)
    const bool small = (int64_t)a.T * per < INT32_MAX;
    const int t = small ? (int)((uint32_t)i / (uint32_t)per) : (int)(i / per), r0 = 4 * (int)(i - (int64_t)t * per);
    int parts = a.parts;
    if (parts == 0) {
        const int blk = (t / a.bm) * a.n_blk + r0 / a.blk_rows;
        parts = run_of((blk + 1) * a.n_slab - 1, a.runs) - run_of(blk * a.n_slab, a.runs) + 1;
    }
    f32x4 sum[N];
#pragma unroll
    for (int l = 0; l < N; ++l) sum[l] = f32x4{0.f, 0.f, 0.f, 0.f};
    const size_t step = (size_t)a.T * N * a.op;
    const float* p = a.partial + ((size_t)t * N) * a.op + r0;
    if (parts <= 2) add_parts<N, 2>(p, step, a.op, parts, sum);
    else if (parts <= 4) add_parts<N, 4>(p, step, a.op, parts, sum);
    else add_parts<N, 8>(p, step, a.op, parts, sum);
    if (a.units != nullptr) {
        const float unit = a.units[t];
#pragma unroll
        for (int l = 0; l < N; ++l)
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[l][r] *= unit;
    }
    float z[N][4], v[4];
#pragma unroll
    for (int l = 0; l < N; ++l)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = min(r0 + r, a.out - 1);
            z[l][r] = a.scales[l] != nullptr ? sum[l][r] * (float)a.scales[l][row] : sum[l][r];
            if (a.bias[l] != nullptr) z[l][r] += (float)a.bias[l][row];
        }
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = z[0][r];
    act_values(a.act, v);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if constexpr (N > 1) v[r] *= z[N - 1][r];
        if (r0 + r >= a.out) break;
        const size_t at = (size_t)t * a.out + r0 + r;
#pragma unroll
        for (int l = 0; l < N; ++l)
            if (a.z[l] != nullptr) a.z[l][at] = (f16)z[l][r];
        if (a.residual != nullptr) v[r] += (float)a.residual[at];
        a.y[at] = (f16)v[r];
    }
}

FinishArgs finish_args(int n, const float* partial, const void* const* scales, const Epilogue& epi, int64_t out,
                       int64_t op, int64_t batch) {
    FinishArgs f = {};
    for (int l = 0; l < n; ++l) {
        f.scales[l] = scales ? static_cast<const f16*>(scales[l]) : nullptr;
        f.bias[l] = static_cast<const f16*>(epi.bias[l]);
        f.z[l] = static_cast<f16*>(epi.z[l]);
    }
    f.partial = partial;
    f.residual = static_cast<const f16*>(epi.residual);
    f.y = static_cast<f16*>(epi.y);
    f.units = epi.units;
    f.out = (int)out;
    f.op = (int)op;
    f.T = (int)batch;
    f.act = epi.act;
    return f;
}

hipError_t launch_finish_args(int n, FinishArgs& f, hipStream_t stream) {
    const int64_t threads = (int64_t)f.T * (f.op / 4), blocks = (threads + 255) / 256;
    const int64_t all = blocks + bias_sum_blocks(f.sums);
    if (all > INT32_MAX) return hipErrorInvalidValue;
    f.blocks = (int)blocks;
    if (n == 2) hipLaunchKernelGGL(skinny_finish_kernel<2>, dim3((unsigned)all), dim3(256), 0, stream, f);
    else hipLaunchKernelGGL(skinny_finish_kernel<1>, dim3((unsigned)all), dim3(256), 0, stream, f);
    return hipGetLastError();
}

// Geometry of one call.
struct SkinnyPlan {
    int bm = 0, blk_rows = 0, op = 0, n_slab = 0, n_blk = 0, slots = 0, half_tile = -1;
    Runs runs = {};
};

// Token tiles of up to 64 tokens for 2x8 (its codebooks leave room for three x stages of
// them), up to 128 for 1x16, which is bound by its gathers, one per code and token tile.
SkinnyPlan skinny_plan(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch) {
    SkinnyPlan p;
    const int64_t bm = batch <= 32 ? 32 : batch <= 64 || sc.B == 8 ? 64 : 128, tile = n == 2 ? 8 : 16;
    const int64_t n_slab = (in / kGroup + kKSlab - 1) / kKSlab, n_blk = (out + kKTiles * tile - 1) / (kKTiles * tile);
    const int64_t units = (batch + bm - 1) / bm * n_blk * n_slab;
    p.bm = (int)bm;
    p.blk_rows = (int)(kKTiles * tile);
    p.op = (int)((out + tile - 1) / tile * tile);
    p.n_slab = (int)n_slab;
    p.n_blk = (int)n_blk;
    const int64_t n_tt = (batch + bm - 1) / bm;
    const bool half = sc.B == 8 && n_tt > 1 && batch - (n_tt - 1) * bm <= bm / 2;
    if (half) p.half_tile = (int)n_tt - 1;
    const int64_t full = (n_tt - 1) * n_blk * n_slab;
    // Two places for a whole unit and one for a half one where that shortens the longest run, a half
    // unit counted as 0.8 (its lookups are whole): 264 units of gated 1000x2733 at 130 tokens, two
    // in some runs, 21.6 -> 16.9 us; 16 a run (4096x11008 at 160) would take 75.1 instead of 71.0.
    int64_t places = units, each = 1;
    if (half) {
        const int64_t q = (full + units + kSkinnyWorkgroups - 1) / kSkinnyWorkgroups;   // places of the longest
        const double weighted = std::max<double>((double)((q + 1) / 2), 0.8 * (double)q);
        if (weighted < (double)((units + kSkinnyWorkgroups - 1) / kSkinnyWorkgroups)) {
            places = full + units;
            each = 2;
        }
    }
    const int64_t W = std::min<int64_t>(kSkinnyWorkgroups, places / each);
    p.runs = Runs{(int)places, (int)W, (int)(places / W), (int)(places % W), each == 2 ? (int)full : -1};
    // the runs that share a row block: those that its slabs fill, and one cut at each end
    p.slots = (int)((each * n_slab * W + places - 1) / places + 1);
    return p;
}

template <int SCHEME, int BM, bool GATED, int RT>
hipError_t launch_main(const SkinnyPlan& p, const SkinnyArgs& a, hipStream_t stream) {
    auto kern = a.G % kKSlab == 0 ? skinny_kernel<SCHEME, BM, GATED, kRowWhole, RT>
                : a.G % 8 == 0    ? skinny_kernel<SCHEME, BM, GATED, kRowVec, RT>
                                  : skinny_kernel<SCHEME, BM, GATED, kRowAny, RT>;
    constexpr size_t lds = (lds_codebooks(SCHEME) ? kKCbBytes : 0) + (size_t)skinny_stages(BM) * BM * kKSlab * 16;
    static_assert(lds <= 163840, "LDS budget");
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(p.runs.W), dim3(64 * kKTiles / RT), lds, stream, a);
    return hipGetLastError();
}

// Up to 32 tokens: one row tile a wave.  Above, the matrix cores and the LDS reads of x weigh
// more than the lookups: two row tiles a wave read x half as often (gated 8192x28672 at 512
// tokens 825 -> 786 us).
template <int SCHEME, bool GATED>
hipError_t launch_scheme(const SkinnyPlan& p, const SkinnyArgs& a, hipStream_t stream) {
    if (p.bm == 32) return launch_main<SCHEME, 32, GATED, 1>(p, a, stream);
    if constexpr (SCHEME == kScheme1x16) {
        if (p.bm == 128) return launch_main<SCHEME, 128, GATED, 2>(p, a, stream);
    }
    return launch_main<SCHEME, 64, GATED, 2>(p, a, stream);
}

}  // namespace

// 1x16: a unit is 131072 gathers, about 9 us of one CU, so few units leave the others idle and decoding the weights
// first is faster (2048x1024 at 64 tokens: 22.2 us against 16.7; 160 units of 4000x2400:
// 26.0 against 29.7), and above 128 tokens every code is gathered twice (4096^2 at 256 tokens, 256 units:
// 46 against 41; 4096x11008, 688 units: 80 against 98; at 512 tokens 128 against 115).  2x8
// wins from the smallest layers (10.9 against 16.4 us on 2048x1024 at 64 tokens) up to 512
// tokens (4096^2 41.7 against 43.5, 11008x4096 87 against 90), gated, whose decoding is spread over twice the
// products, up to about 384 (4096x11008 136 against 152, 8192x28672 608 against 580; at 512 178 against 169 and
// 805 against 676).  4x8 g16 wins likewise (1024^2 at 17 tokens 9.8 us against 13.3, gated 4096x11008 at 64 49
// against 140) up to about 320 (11008x4096 92.7 against 96.8), gated 256 (4096x11008 150 against 148, at 320 both 181).
bool skinny_serves(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch) {
    const bool two = sc.M == 2 && sc.B == 8 && sc.g == 8, one = sc.M == 1 && sc.B == 16 && sc.g == 8;
    const bool four = sc.M == 4 && sc.B == 8 && sc.g == 16;
    if (!two && !one && !four) return false;
    if (out * (in / kGroup) < 8) return false;   // 16 bytes of codes a load
    if (batch > skinny_max_batch(sc, n)) return false;
    const int64_t rows = kKTiles * (n == 2 ? 8 : 16);
    const int64_t units = (out + rows - 1) / rows * ((in / kGroup + kKSlab - 1) / kKSlab);
    if (one && units < (batch <= kSkinnyMaxBatch1x16Few ? 128 : 512)) return false;
    return (batch + 31) / 32 * units < (1 << 30);   // units are counted in 32 bits
}

int64_t skinny_partial_bytes(const GenericScheme& sc, int n, int64_t out, int64_t in, int64_t batch) {
    // the plan changes at multiples of 32 tokens and is linear in the batch in between
    int64_t room = 0;
    for (int64_t t = std::min<int64_t>(32, batch);; t = std::min(t + 32, batch)) {
        const SkinnyPlan p = skinny_plan(sc, n, out, in, t);
        room = std::max(room, (int64_t)p.slots * t * n * p.op * 4);
        if (t == batch) return room;
    }
}

hipError_t launch_skinny(const GenericScheme& sc, const ActLayers& L, const void* x, void* partial, const Epilogue& epi,
                         int64_t out, int64_t in, int64_t batch, hipStream_t stream) {
    const SkinnyPlan p = skinny_plan(sc, L.n, out, in, batch);
    SkinnyArgs a = {};
    for (int l = 0; l < L.n; ++l) {
        a.codes[l] = static_cast<const uint8_t*>(L.codes[l]);
        a.codebooks[l] = static_cast<const f16*>(L.codebooks[l]);
    }
    a.x = static_cast<const f16*>(x);
    a.partial = static_cast<float*>(partial);
    a.out = (int)out;
    a.op = p.op;
    a.G = (int)(in / kGroup);
    a.T = (int)batch;
    FinishArgs f = finish_args(L.n, a.partial, L.scales, epi, out, p.op, batch);
    f.n_slab = a.n_slab = p.n_slab;
    f.n_blk = a.n_blk = p.n_blk;
    f.runs = a.runs = p.runs;
    a.half_tile = p.half_tile;
    f.bm = p.bm;
    f.blk_rows = p.blk_rows;
    const bool gated = L.n == 2;
    const hipError_t e = sc.M == 2   ? (gated ? launch_scheme<kScheme2x8, true>(p, a, stream) : launch_scheme<kScheme2x8, false>(p, a, stream))
                         : sc.M == 1 ? (gated ? launch_scheme<kScheme1x16, true>(p, a, stream) : launch_scheme<kScheme1x16, false>(p, a, stream))
                                     : (gated ? launch_scheme<kSchemeB8M4, true>(p, a, stream) : launch_scheme<kSchemeB8M4, false>(p, a, stream));
    if (e != hipSuccess) return e;
    return launch_finish_args(L.n, f, stream);
}

hipError_t launch_finish(int n, const float* partial, const void* const* scales, const Epilogue& epi, int64_t out,
                         int64_t op, int64_t batch, int parts, const BiasSum& bias, hipStream_t stream) {
    FinishArgs f = finish_args(n, partial, scales, epi, out, op, batch);
    f.sums = bias;
    f.parts = parts;
    return launch_finish_args(n, f, stream);
}

}  // namespace aqlm
