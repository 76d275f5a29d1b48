// Products of MX4 weights with many tokens: z[t][i] = sum_k W[i][k] x[t][k], then mx4_linear.hip's epilogue.
//
// The scaled matrix instructions take codes and scales as they are, so the work is to bring them on time.  A workgroup of 8
// waves owns a tile of TM rows of W x TN tokens; wave (m, n) of WM x WN a part of MT x NT squares of 32 x 32, which
// each take one instruction a step of 64 inputs (four with x split in pieces).  Inputs pass through LDS in stages of 128, loaded
// straight from memory, with one barrier a stage; the two waves of a SIMD read and multiply in turn.
//
// LDS of a stage:
//   rows of MX4 (W, and x where it is MX4): 64 bytes a row; block b of row r lies in slot b ^ (r / 4 % 4), so that the 16 lanes
//     that one clock of a 16-byte read serves (0-3, 12-15, 20-27; 4-11, 16-19, 28-31; likewise above 32) find 16 distinct
//     banks, and four neighbouring lanes of a load still read 64 contiguous bytes;
//   split x: the records of mx4.h as they are.
// Scale bytes of MX4 rows: 16 bytes a row at a time, four stages' worth, from any address, through registers into LDS of their
// own (two buffers).  A lane reads the four bytes of its row and stage and moves its half of the wave's to where the
// instruction's byte selection finds it.
//
// LDS reads are inline assembly with their wait, because the compiler would make every LDS read wait for the
// loads into LDS that are still in flight.
#include <algorithm>

#include "act_bias.h"
#include "act_math.h"
#include "mx4_gemm.h"

namespace aqlm {

namespace {

constexpr int kThreads = 512, kWaves = 8;
constexpr int kStageBlocks = 4;        // blocks of a stage: 128 inputs
constexpr int kScaleStages = 4;        // stages that a load of scales serves

struct GemmArgs {
    const uint8_t* w;        // codes, scales of W
    const uint8_t* ws;
    const uint8_t* x;        // codes, scales of x; or its split records (xs NULL)
    const uint8_t* xs;
    const f16* bias;
    const f16* residual;     // may be y
    f16* y;
    float* part;             // [split][token][op], for splits > 1
    int act, out, T, nb, op;
    int tiles_m, tiles_n, splits, stages;   // stages of the whole row; of a split: a multiple of kScaleStages
};

template <int FMT, int WM, int WN, int MT, int NT, int STAGES>
struct Tile {
    static constexpr int kM = WM * MT * 32, kN = WN * NT * 32;
    static constexpr int kABytes = kM * 64;
    static constexpr int kBBytes = FMT == kFmt4 ? kN * 64 : kN / 32 * kStageBlocks * kSplitRecord;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kScaleRows = kM + (FMT == kFmt4 ? kN : 0);
    static constexpr int kScales = STAGES * kStage;                        // their place in LDS
    static constexpr int kPipe = kScales + 2 * kScaleRows * 16;
    static constexpr int kEpiRow = MT * 32 * 4 + 16;                       // bytes of a token's row of a wave's epilogue tile
    static constexpr int kLds = kPipe > kWaves * 32 * kEpiRow ? kPipe : kWaves * 32 * kEpiRow;
    static constexpr int kLoads = (kStage / 1024 + (kStage % 1024 != 0) + kWaves - 1) / kWaves;   // a wave, a stage
    static_assert(WM * WN == kWaves && kLds <= 163840 && kScaleRows <= kThreads);
    static_assert(kStage % 1024 == 0, "whole loads of a wave");
};

// 16 bytes of an array of `total` >= 16 from any offset; bytes past its end are zero.
__device__ __forceinline__ u32x4 load_bytes16(const uint8_t* __restrict__ p, int64_t at, int64_t total) {
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
    const int64_t from = at < total - 16 ? at : total - 16;
    const u32x4_any v = *reinterpret_cast<const u32x4_any*>(p + from);
    u32x4 r = {v[0], v[1], v[2], v[3]};
    const int d = (int)(at - from < 16 ? at - from : 16);
    if (d & 1) r = u32x4{(uint32_t)__builtin_amdgcn_alignbyte(r[1], r[0], 1), (uint32_t)__builtin_amdgcn_alignbyte(r[2], r[1], 1),
                         (uint32_t)__builtin_amdgcn_alignbyte(r[3], r[2], 1), r[3] >> 8};
    if (d & 2) r = u32x4{(uint32_t)__builtin_amdgcn_alignbyte(r[1], r[0], 2), (uint32_t)__builtin_amdgcn_alignbyte(r[2], r[1], 2),
                         (uint32_t)__builtin_amdgcn_alignbyte(r[3], r[2], 2), r[3] >> 16};
    if (d & 4) r = u32x4{r[1], r[2], r[3], 0u};
    if (d & 8) r = u32x4{r[2], r[3], 0u, 0u};
    if (d & 16) r = u32x4{0u, 0u, 0u, 0u};
    return r;
}

__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)lds_ptr(const_cast<void*>(p)); }

// One step of 64 inputs: the operands of MT row squares, from `a` + 2048 i.
template <int MT>
struct AOperand {
    u32x4 v[MT];
};


// Reads of a wave's operands, all waited for.  a: LDS address of the lane's block of the first row square; b: of x.
__device__ __forceinline__ void read_4(AOperand<4>& a, u32x4 (&b)[2], uint32_t pa, uint32_t pb) {
    asm volatile("ds_read_b128 %0, %6\n\tds_read_b128 %1, %6 offset:2048\n\tds_read_b128 %2, %6 offset:4096\n\t"
                 "ds_read_b128 %3, %6 offset:6144\n\tds_read_b128 %4, %7\n\tds_read_b128 %5, %7 offset:2048\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(a.v[0]), "=&v"(a.v[1]), "=&v"(a.v[2]), "=&v"(a.v[3]), "=&v"(b[0]), "=&v"(b[1])
                 : "v"(pa), "v"(pb)
                 : "memory");
}
__device__ __forceinline__ void read_4(AOperand<2>& a, u32x4 (&b)[1], uint32_t pa, uint32_t pb) {
    asm volatile("ds_read_b128 %0, %3\n\tds_read_b128 %1, %3 offset:2048\n\tds_read_b128 %2, %4\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(a.v[0]), "=&v"(a.v[1]), "=&v"(b[0])
                 : "v"(pa), "v"(pb)
                 : "memory");
}
// x in pieces: the first 16 bytes of piece p at pb + 512 p, the other 8 at pr + 256 p, the scale word at ps.
__device__ __forceinline__ void read_6(AOperand<4>& a, u32x4 (&b)[4], u32x2 (&r)[4], uint32_t& s, uint32_t pa, uint32_t pb,
                                       uint32_t pr, uint32_t ps) {
    asm volatile("ds_read_b128 %0, %13\n\tds_read_b128 %1, %13 offset:2048\n\tds_read_b128 %2, %13 offset:4096\n\t"
                 "ds_read_b128 %3, %13 offset:6144\n\t"
                 "ds_read_b128 %4, %14\n\tds_read_b128 %5, %14 offset:512\n\tds_read_b128 %6, %14 offset:1024\n\t"
                 "ds_read_b128 %7, %14 offset:1536\n\t"
                 "ds_read_b64 %8, %15\n\tds_read_b64 %9, %15 offset:256\n\tds_read_b64 %10, %15 offset:512\n\t"
                 "ds_read_b64 %11, %15 offset:768\n\tds_read_b32 %12, %16\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(a.v[0]), "=&v"(a.v[1]), "=&v"(a.v[2]), "=&v"(a.v[3]), "=&v"(b[0]), "=&v"(b[1]), "=&v"(b[2]), "=&v"(b[3]),
                   "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(s)
                 : "v"(pa), "v"(pb), "v"(pr), "v"(ps)
                 : "memory");
}
__device__ __forceinline__ void read_6(AOperand<2>& a, u32x4 (&b)[4], u32x2 (&r)[4], uint32_t& s, uint32_t pa, uint32_t pb,
                                       uint32_t pr, uint32_t ps) {
    asm volatile("ds_read_b128 %0, %11\n\tds_read_b128 %1, %11 offset:2048\n\t"
                 "ds_read_b128 %2, %12\n\tds_read_b128 %3, %12 offset:512\n\tds_read_b128 %4, %12 offset:1024\n\t"
                 "ds_read_b128 %5, %12 offset:1536\n\t"
                 "ds_read_b64 %6, %13\n\tds_read_b64 %7, %13 offset:256\n\tds_read_b64 %8, %13 offset:512\n\t"
                 "ds_read_b64 %9, %13 offset:768\n\tds_read_b32 %10, %14\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(a.v[0]), "=&v"(a.v[1]), "=&v"(b[0]), "=&v"(b[1]), "=&v"(b[2]), "=&v"(b[3]), "=&v"(r[0]), "=&v"(r[1]),
                   "=&v"(r[2]), "=&v"(r[3]), "=&v"(s)
                 : "v"(pa), "v"(pb), "v"(pr), "v"(ps)
                 : "memory");
}
// N scale words, 512 bytes (32 rows) apart.
__device__ __forceinline__ void read_scales(uint32_t (&s)[4], uint32_t p) {
    asm volatile("ds_read_b32 %0, %4\n\tds_read_b32 %1, %4 offset:512\n\tds_read_b32 %2, %4 offset:1024\n\t"
                 "ds_read_b32 %3, %4 offset:1536\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(s[0]), "=&v"(s[1]), "=&v"(s[2]), "=&v"(s[3])
                 : "v"(p)
                 : "memory");
}
__device__ __forceinline__ void read_scales(uint32_t (&s)[2], uint32_t p) {
    asm volatile("ds_read_b32 %0, %2\n\tds_read_b32 %1, %2 offset:512\n\ts_waitcnt lgkmcnt(0)" : "=&v"(s[0]), "=&v"(s[1]) : "v"(p) : "memory");
}
__device__ __forceinline__ void read_scales(uint32_t (&s)[1], uint32_t p) {
    asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(s[0]) : "v"(p) : "memory");
}

template <int FMT, int WM, int WN, int MT, int NT, int STAGES, bool PART>
__global__ __launch_bounds__(kThreads) void mx4_gemm_kernel(GemmArgs g) {
    using L = Tile<FMT, WM, WN, MT, NT, STAGES>;
    extern __shared__ u32x4 smem[];
    char* lds = reinterpret_cast<char*>(smem);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int l32 = lane & 31, half = lane >> 5;
    // tokens fastest: an XCD's workgroups share rows of W
    const int u = xcd_run((int)blockIdx.x, (int)gridDim.x);
    const int n0 = u % g.tiles_n * L::kN, m0 = u / g.tiles_n % g.tiles_m * L::kM, split = u / g.tiles_n / g.tiles_m;
    const int per = ((g.stages + g.splits - 1) / g.splits + kScaleStages - 1) / kScaleStages * kScaleStages;
    const int first = split * per, n_stage = min(per, g.stages - first);
    const int nb = g.nb;
    const int wm = wave / WN, wn = wave % WN;

    // Load j of this wave in a stage: 64 chunks of 16 bytes, from `chunk` on.  Loads past the stage repeat the last.
    auto load_stage = [&](int s) {
        char* to = lds + s % STAGES * L::kStage;
        const int b0 = (first + s) * kStageBlocks;
#pragma unroll
        for (int j = 0; j < L::kLoads; ++j) {
            const int i = min(wave + j * kWaves, L::kStage / 1024 - 1);   // uniform
            const int c = i * 64 + lane;
            const void* from;
            if (i < L::kABytes / 1024) {
                const int r = c / 4, b = b0 + ((c & 3) ^ ((r >> 2) & 3));
                from = g.w + ((size_t)min(m0 + r, g.out - 1) * nb + min(b, nb - 1)) * kMxBlockBytes;
            } else if constexpr (FMT == kFmt4) {
                const int cb = c - L::kABytes / 16, r = cb / 4, b = b0 + ((cb & 3) ^ ((r >> 2) & 3));
                from = g.x + ((size_t)min(n0 + r, g.T - 1) * nb + min(b, nb - 1)) * kMxBlockBytes;
            } else {
                constexpr int kPer = kSplitRecord / 16;   // chunks of a record
                const int cb = c - L::kABytes / 16, rec = cb / kPer, tile = rec / kStageBlocks;
                const int tt = min(n0 / kSplitTokens + tile, (g.T - 1) / kSplitTokens);
                from = g.x + ((size_t)tt * nb + min(b0 + rec % kStageBlocks, nb - 1)) * kSplitRecord + (cb % kPer) * 16;
            }
            __builtin_amdgcn_global_load_lds(from, lds_ptr(to + i * 1024), 16, 0, 0);
        }
    };
    // Scales of four stages: thread r has row r of W, then of x.
    const bool has_scales = tid < L::kScaleRows;
    auto load_scales = [&](int c) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (has_scales) {
            const bool of_w = tid < L::kM;
            const int row = of_w ? min(m0 + tid, g.out - 1) : min(n0 + tid - L::kM, g.T - 1);
            v = load_bytes16(of_w ? g.ws : g.xs, (int64_t)row * nb + (int64_t)(first + c * kScaleStages) * kStageBlocks,
                             (int64_t)(of_w ? g.out : g.T) * nb);
        }
        return v;
    };
    auto keep_scales = [&](u32x4 v, int c) {
        if (has_scales) {
            const uint32_t at = lds_address(lds + L::kScales + (c & 1) * L::kScaleRows * 16 + tid * 16);
            asm volatile("ds_write_b128 %0, %1" ::"v"(at), "v"(v) : "memory");
        }
    };

    f32x16 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x16{};

    u32x4 sc = load_scales(0);
    keep_scales(sc, 0);
    sc = load_scales(1);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < n_stage) load_stage(s);

    // LDS addresses of the lane's operands in a stage
    const uint32_t lds0 = lds_address(lds);
    const uint32_t fold = (lane >> 2) & 3;
    const uint32_t pa = (uint32_t)(wm * MT * 32 + l32) * 64 + ((half ^ fold) * 16);   // second step: bit 5 flipped
    const uint32_t pb4 = L::kABytes + (uint32_t)(wn * NT * 32 + l32) * 64 + ((half ^ fold) * 16);
    const uint32_t pb6 = L::kABytes + (uint32_t)(wn * NT * kStageBlocks + half) * kSplitRecord;
    const uint32_t sa0 = lds0 + L::kScales + (uint32_t)(wm * MT * 32 + l32) * 16;
    const uint32_t sb0 = lds0 + L::kScales + (uint32_t)(L::kM + wn * NT * 32 + l32) * 16;

    for (int s = 0; s < n_stage; ++s) {
        // this wave's loads of stage s have landed (those of the STAGES - 2 behind it may be in flight), and the barrier says
        // so for all; every wave has read stage s - 1, whose place is loaded next
        if (s + STAGES - 1 <= n_stage)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(L::kLoads * (STAGES - 2)) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (s + STAGES - 1 < n_stage) load_stage(s + STAGES - 1);
        const int c = s / kScaleStages;
        if (s % kScaleStages == kScaleStages - 1) {
            keep_scales(sc, c + 1);
            sc = load_scales(c + 2);
        }
        const uint32_t base = lds0 + s % STAGES * L::kStage;
        const uint32_t soff = (c & 1) * L::kScaleRows * 16 + s % kScaleStages * 4;
        uint32_t sa[MT], sb[NT];
        read_scales(sa, sa0 + soff);
#pragma unroll
        for (int i = 0; i < MT; ++i) sa[i] >>= 8 * half;
        if constexpr (FMT == kFmt4) {
            read_scales(sb, sb0 + soff);
#pragma unroll
            for (int j = 0; j < NT; ++j) sb[j] >>= 8 * half;
        }
        const int b0 = (first + s) * kStageBlocks + half;
        const bool whole = (first + s + 1) * kStageBlocks <= nb;   // uniform
        auto step = [&](auto ks_const) {
            constexpr int KS = decltype(ks_const)::value;
            AOperand<MT> a;
            u32x4 b4[NT], b[4];
            u32x2 r[4];
            uint32_t s6;
            const uint32_t flip = KS * 32;
            if constexpr (FMT == kFmt4) {
                read_4(a, b4, (base + pa) ^ flip, (base + pb4) ^ flip);
            } else {
                const uint32_t q = base + pb6 + KS * 2 * kSplitRecord;
                read_6(a, b, r, s6, (base + pa) ^ flip, q + l32 * 16, q + 2048 + l32 * 8, q + 3072 + l32 * 4);
            }
            if (!whole) {   // blocks past the row: codes 0 and scales of 1, whatever was loaded
                const bool in_row = b0 + 2 * KS < nb;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    a.v[i] = in_row ? a.v[i] : u32x4{0u, 0u, 0u, 0u};
                    sa[i] = in_row ? sa[i] : 0x7f7f7f7fu;
                }
                if constexpr (FMT == kFmt4) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) sb[j] = in_row ? sb[j] : 0x7f7f7f7fu;
                }
            }
            if constexpr (FMT == kFmt4) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        acc[i][j] = mfma_mx32<kFmt4, 2 * KS, 2 * KS>(operand4(a.v[i]), operand4(b4[j]), acc[i][j], sa[i], sb[j]);
            } else {
                auto piece = [&](int p) { return operand6(u32x6{b[p][0], b[p][1], b[p][2], b[p][3], r[p][0], r[p][1]}); };
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[i][0] = mfma_mx32<kFmt6, 2 * KS, 3>(operand4(a.v[i]), piece(3), acc[i][0], sa[i], s6);
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[i][0] = mfma_mx32<kFmt6, 2 * KS, 2>(operand4(a.v[i]), piece(2), acc[i][0], sa[i], s6);
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[i][0] = mfma_mx32<kFmt6, 2 * KS, 1>(operand4(a.v[i]), piece(1), acc[i][0], sa[i], s6);
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[i][0] = mfma_mx32<kFmt6, 2 * KS, 0>(operand4(a.v[i]), piece(0), acc[i][0], sa[i], s6);
            }
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
    }

    // Epilogue: a wave turns its squares in LDS of its own (token rows of MT * 32 floats, 16 bytes apart), and a lane finishes
    // four neighbouring outputs of a token.
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) pin(acc[i][j]);
    __syncthreads();
    char* turn = lds + wave * 32 * L::kEpiRow;
    constexpr int kQuads = MT * 8;   // lanes a token
    const int row = m0 + wm * MT * 32 + 4 * (lane % kQuads);
    const bool vec = g.out % 4 == 0;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (!PART && g.bias != nullptr) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (row + q < g.out) bias[q] = (float)g.bias[row + q];
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(turn + l32 * L::kEpiRow + (i * 32 + 8 * q + 4 * half) * 4) =
                    f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t0 = 0; t0 < 32; t0 += 64 / kQuads) {
            const int t = t0 + lane / kQuads, token = n0 + (wn * NT + j) * 32 + t;
            const f32x4 z = *reinterpret_cast<const f32x4*>(turn + t * L::kEpiRow + (lane % kQuads) * 16);
            if (token >= g.T) continue;
            if constexpr (PART) {
                if (row < g.op) *reinterpret_cast<f32x4*>(g.part + ((size_t)split * g.T + token) * g.op + row) = z;
            } else {
                if (row >= g.out) continue;
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = z[q] + bias[q];
                act_values(g.act, v);
                const size_t at = (size_t)token * g.out + row;
                typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
                if (vec) {
                    if (g.residual != nullptr) {
                        const f16x4 res = *reinterpret_cast<const f16x4*>(g.residual + at);
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] += (float)res[q];
                    }
                    *reinterpret_cast<f16x4*>(g.y + at) = f16x4{(f16)v[0], (f16)v[1], (f16)v[2], (f16)v[3]};
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (row + q < g.out) {
                            if (g.residual != nullptr) v[q] += (float)g.residual[at + q];
                            g.y[at + q] = (f16)v[q];
                        }
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

struct GemmPlan {
    bool big;
    int tiles_m, tiles_n, splits;
};

template <int FMT, int WM, int WN, int MT, int NT, int STAGES>
hipError_t launch_tile(GemmArgs& g, hipStream_t stream) {
    using L = Tile<FMT, WM, WN, MT, NT, STAGES>;
    g.tiles_m = (g.out + L::kM - 1) / L::kM;
    g.tiles_n = (g.T + L::kN - 1) / L::kN;
    auto kern = g.splits > 1 ? mx4_gemm_kernel<FMT, WM, WN, MT, NT, STAGES, true> : mx4_gemm_kernel<FMT, WM, WN, MT, NT, STAGES, false>;
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, L::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)g.tiles_m * g.tiles_n * g.splits)), dim3(kThreads), L::kLds, stream, g);
    return hipGetLastError();
}

int64_t round4(int64_t v) { return (v + 3) / 4 * 4; }

// The small tile (128 x 128) and how many parts of the sum fill the chip with it.
constexpr int kSmall = 128, kWant = 512;
int max_splits(int64_t in) { return (int)std::max<int64_t>(1, in / (2 * kScaleStages * kStageBlocks * kMxBlock)); }

GemmPlan gemm_plan(bool x_mx4, int64_t out, int64_t in, int64_t batch) {
    const int64_t big_n = x_mx4 ? 256 : 128;
    GemmPlan p;
    const int64_t big = (out + 255) / 256 * ((batch + big_n - 1) / big_n);
    p.big = big >= 192;
    p.tiles_m = (int)((out + kSmall - 1) / kSmall);
    p.tiles_n = (int)((batch + kSmall - 1) / kSmall);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    p.splits = p.big ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(max_splits(in), 256 / tiles));
    // no empty part
    const int64_t stages = (in / kMxBlock + kStageBlocks - 1) / kStageBlocks;
    while (p.splits > 1) {
        const int64_t per = ((stages + p.splits - 1) / p.splits + kScaleStages - 1) / kScaleStages * kScaleStages;
        if (per * (p.splits - 1) < stages) break;
        --p.splits;
    }
    return p;
}

}  // namespace

bool mx4_gemm_serves(int64_t out, int64_t in, int64_t batch) {
    return batch > 64 && out * (in / kMxBlock) >= 16;   // load_bytes16's least array
}

int64_t mx4_gemm_part_bytes(int64_t out, int64_t in, int64_t batch) {
    // splits <= max_splits and splits * tiles_n <= kWant / tiles_m: the most of any batch up to this one
    const int64_t tiles_m = (out + kSmall - 1) / kSmall, cap = std::max<int64_t>(1, kWant / tiles_m) * kSmall;
    return max_splits(in) < 2 ? 0 : std::min(max_splits(in) * batch, cap) * round4(out) * (int64_t)sizeof(float);
}

hipError_t launch_mx4_gemm(const void* codes, const void* scales, MxInput x, const Epilogue& e, void* part, int64_t out, int64_t in,
                           int64_t batch, hipStream_t stream) {
    const GemmPlan p = gemm_plan(x.scales != nullptr, out, in, batch);
    GemmArgs g = {};
    g.w = static_cast<const uint8_t*>(codes);
    g.ws = static_cast<const uint8_t*>(scales);
    g.x = static_cast<const uint8_t*>(x.x);
    g.xs = static_cast<const uint8_t*>(x.scales);
    g.bias = static_cast<const f16*>(e.bias[0]);
    g.residual = static_cast<const f16*>(e.residual);
    g.y = static_cast<f16*>(e.y);
    g.part = static_cast<float*>(part);
    g.act = e.act;
    g.out = (int)out;
    g.T = (int)batch;
    g.nb = (int)(in / kMxBlock);
    g.op = (int)round4(out);
    g.splits = p.splits;
    g.stages = (g.nb + kStageBlocks - 1) / kStageBlocks;
    hipError_t r;
    if (x.scales != nullptr) r = p.big ? launch_tile<kFmt4, 2, 4, 4, 2, 4>(g, stream) : launch_tile<kFmt4, 2, 4, 2, 1, 4>(g, stream);
    else r = p.big ? launch_tile<kFmt6, 2, 4, 4, 1, 2>(g, stream) : launch_tile<kFmt6, 2, 4, 2, 1, 2>(g, stream);
    if (r != hipSuccess || p.splits == 1) return r;
    return launch_finish(1, g.part, nullptr, e, out, g.op, batch, p.splits, BiasSum{}, stream);
}

}  // namespace aqlm
